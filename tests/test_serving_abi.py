"""Refusals of the serving operators, on the CPU: every case fails the synchronous checks, before any launch."""
import ctypes

import pytest
import torch

from lm_causal_depthwise_b200 import api, build

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def _p(n):
    return ctypes.c_void_p(n) if n else None


def _norm(lib, M=4, N=512, group=0, x=MB, r=2 * MB, w=3 * MB, eps=1e-6, ro=4 * MB, out=5 * MB, sc=6 * MB):
    if group == 0:
        return lib.rglru_add_rmsnorm(M, N, _p(x), _p(r), _p(w), eps, _p(ro), _p(out), None)
    return lib.rglru_add_rmsnorm_e4m3(M, N, group, _p(x), _p(r), _p(w), eps, _p(ro), _p(out), _p(sc), None)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("kw", [dict(M=0), dict(N=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(x=0),
                                dict(w=0), dict(out=0), dict(x=MB + 8), dict(out=5 * MB + 2), dict(r=0), dict(ro=0),
                                dict(out=MB), dict(out=2 * MB), dict(out=4 * MB), dict(ro=MB + 16), dict(ro=3 * MB),
                                dict(ro=2 * MB + 512)])
def test_norm_refuses(lib, group, kw):
    assert _norm(lib, group=group, **kw) == api.ERR_INVALID_ARG


def test_norm_refuses_sizes_and_groups(lib):
    for N in (12, 16392):
        assert _norm(lib, N=N) == api.ERR_UNSUPPORTED
    for N, g in ((512, 16), (512, 48), (512, 512), (160, 64), (512, -32)):
        assert _norm(lib, N=N, group=g) == api.ERR_UNSUPPORTED
    assert lib.rglru_add_rmsnorm_e4m3(4, 512, 0, _p(MB), None, _p(MB), 1e-6, None, _p(MB), _p(MB), None) \
        == api.ERR_UNSUPPORTED
    assert _norm(lib, group=64, sc=0) == api.ERR_INVALID_ARG
    assert _norm(lib, group=64, sc=MB) == api.ERR_INVALID_ARG
    assert _norm(lib, group=64, sc=5 * MB) == api.ERR_INVALID_ARG


def _w4(lib, M=3, N=100, K=256, group=64, A=MB, As=0, ag=0, W=2 * MB, Ws=3 * MB, b=4 * MB, out=5 * MB):
    return lib.rglru_linear_w4(M, N, K, group, _p(A), _p(As), ag, _p(W), _p(Ws), _p(b), _p(out), None)


@pytest.mark.parametrize("kw,st", [
    (dict(M=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(M=65), 2), (dict(group=16), 2), (dict(group=256), 2),
    (dict(K=96, group=64), 2), (dict(As=6 * MB, ag=48), 2), (dict(As=6 * MB, ag=0), 2),
    (dict(As=6 * MB, ag=128, K=192), 2), (dict(K=1 << 21), 2), (dict(A=0), 1), (dict(W=0), 1), (dict(Ws=0), 1),
    (dict(out=0), 1), (dict(A=MB + 4), 1), (dict(b=4 * MB + 4), 1), (dict(As=6 * MB + 4, ag=64), 1), (dict(out=MB), 1),
    (dict(out=2 * MB), 1), (dict(out=3 * MB), 1), (dict(out=4 * MB), 1), (dict(As=5 * MB, ag=64), 1)])
def test_linear_w4_refuses(lib, kw, st):
    assert _w4(lib, **kw) == st


NAMES = ("qkv", "cu", "ctx", "table", "q", "k", "ks", "v", "vs", "ws")


def _paged(lib, attend, rows=8, S=2, H=4, Hkv=2, D=128, page=16, pages=8, max_pages=4, max_new=4, max_total=64,
           window=32, scale=0.1, base=10000.0, wsb=None, **ptr):
    at = {n: 16 * MB * (i + 1) for i, n in enumerate(NAMES)}
    at.update(ptr)
    a = {n: _p(v) for n, v in at.items()}
    if attend:
        need = lib.rglru_paged_attention_workspace_size(H, Hkv, D) or 1 << 20
        return lib.rglru_paged_attention(rows, S, H, Hkv, D, page, pages, max_pages, max_new, max_total, window, scale,
                                         a["qkv"], a["cu"], a["ctx"], a["table"], a["k"], a["ks"], a["v"], a["vs"],
                                         a["q"], a["ws"], need if wsb is None else wsb, None)
    return lib.rglru_paged_append(rows, S, H, Hkv, D, page, pages, max_pages, max_new, max_total, a["qkv"], a["cu"],
                                  a["ctx"], a["table"], base, a["q"], a["k"], a["ks"], a["v"], a["vs"], a["ws"],
                                  4096 if wsb is None else wsb, None)


@pytest.mark.parametrize("attend", [False, True])
@pytest.mark.parametrize("kw,st", [
    (dict(rows=0), 1), (dict(S=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(max_pages=0), 1),
    (dict(max_new=0), 1), (dict(max_total=3), 1), (dict(max_total=65), 1), (dict(D=64), 2), (dict(D=512), 2),
    (dict(page=8), 2), (dict(page=24), 2), (dict(page=256), 2), (dict(S=70000), 2), (dict(H=3), 2), (dict(H=257, Hkv=1), 2),
    (dict(H=130, Hkv=65), 2), (dict(rows=1 << 25), 2), (dict(max_total=(1 << 30) + 1, max_pages=1 << 27), 2),
    (dict(wsb=16), 3), (dict(ws=0), 3), (dict(ws=8), 3)]
    + [(dict([(n, 0)]), 1) for n in NAMES[:-1]] + [(dict([(n, 8)]), 1) for n in NAMES[:-1]]
    + [(dict([(n, 16 * MB * 5)]), 1) for n in NAMES if n != "q"] + [(dict(ws=16 * MB * (NAMES.index("k") + 1)), 1)])
def test_paged_calls_refuse(lib, attend, kw, st):
    assert _paged(lib, attend, **kw) == st


def test_paged_calls_refuse_their_own(lib):
    for base in (1.0, 0.0, -5.0, float("nan"), float("inf")):
        assert _paged(lib, False, base=base) == api.ERR_INVALID_ARG
    # k over v: append writes both
    assert _paged(lib, False, k=16 * MB * (NAMES.index("v") + 1)) == api.ERR_INVALID_ARG
    assert _paged(lib, True, window=0) == api.ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _paged(lib, True, scale=scale) == api.ERR_INVALID_ARG
    for H, Hkv, D in ((0, 1, 128), (4, 3, 128), (4, 1, 64), (257, 1, 128), (4, 0, 256)):
        assert lib.rglru_paged_attention_workspace_size(H, Hkv, D) == 0
    assert lib.rglru_paged_attention_workspace_size(10, 1, 256) >= 4096


def _batch(**kw):
    b = dict(cu_tokens=torch.zeros(3, dtype=torch.int32), ctx_len=torch.zeros(2, dtype=torch.int32),
             block_table=torch.zeros(2, 4, dtype=torch.int32), max_new=1, max_total=64)
    b.update(kw)
    return api.PagedBatch(**b)


def test_binding_refuses(lib):
    """Types, shapes, contiguity and host tensors raise in the binding."""
    bf = torch.bfloat16
    x, w = torch.zeros(4, 256, dtype=bf), torch.ones(256)
    with pytest.raises(ValueError, match="CUDA"):
        api.add_rmsnorm(x, x, w)
    with pytest.raises(TypeError):
        api.add_rmsnorm(x.float(), x, w)
    with pytest.raises(ValueError):
        api.add_rmsnorm(x, x[:2], w)
    with pytest.raises(ValueError):
        api.add_rmsnorm(x[:0], None, w)
    with pytest.raises(ValueError):
        api.add_rmsnorm(x, None, w, residual_out=x)
    with pytest.raises(ValueError):
        api.add_rmsnorm(torch.zeros(256, 4, dtype=bf).t(), None, w)
    with pytest.raises(ValueError):
        api.add_rmsnorm_e4m3(x, None, w, group=96)
    W, s = torch.zeros(8, 128, dtype=torch.uint8), torch.ones(8, 4, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_w4(x, W, s)
    with pytest.raises(ValueError):
        api.linear_w4(x, W[:, :64], s)
    with pytest.raises(TypeError):
        api.linear_w4(x, W, s.float())
    with pytest.raises(ValueError):
        api.linear_w4(x, W, torch.ones(8, 3, dtype=bf))
    with pytest.raises(TypeError):
        api.linear_w4(x, W, s, A_scale=torch.ones(4, 2))      # bf16 values with 8-bit scales
    with pytest.raises(ValueError):
        api.linear_w4(x[:0], W, s)
    cache = api.paged_cache(8, 2, 16, 128, device="cpu")
    qkv = torch.zeros(2, 8 * 128, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        api.paged_append(qkv, _batch(), cache, workspace=torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError):
        api.paged_append(qkv[:, :4 * 128], _batch(), cache)   # no query head left
    with pytest.raises(ValueError):
        api.paged_append(qkv, _batch(cu_tokens=torch.zeros(2, dtype=torch.int32)), cache)
    with pytest.raises(TypeError):
        api.paged_append(qkv, _batch(block_table=torch.zeros(2, 4, dtype=torch.int64)), cache)
    with pytest.raises(ValueError, match="CUDA"):
        api.paged_attention(qkv[:, :512].contiguous(), _batch(), cache, workspace=torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        api.paged_attention(qkv[:, :500].contiguous(), _batch(), cache)
    with pytest.raises(api.RGLRUError):
        api.paged_attention_workspace_size(4, 3, 128)


def test_the_block_form_reaches_the_same_checks(lib):
    """rglru_serving_call: each parameter arrives in its place (its own refusal), unknown calls and no block are refused."""
    call = lib.rglru_serving_call
    assert call(5, b"\0" * 256) == call(-1, b"\0" * 256) == call(0, None) == api.ERR_INVALID_ARG

    def tries(name, good, cases):
        k, pack = api._CALLS[name]
        assert call(k, pack(*good.values())) == good_status
        for key, value, st in cases:
            assert key in good
            assert call(k, pack(*{**good, key: value}.values())) == st, (name, key)

    # a size of zero first: nothing is launched, and every later refusal of its own status shows its place
    good_status = api.ERR_UNSUPPORTED
    norm = dict(M=4, N=12, x=MB, r=2 * MB, w=3 * MB, eps=1e-6, ro=4 * MB, out=5 * MB, stream=0)
    tries("rglru_add_rmsnorm", norm, [("M", 0, 1), ("eps", 0.0, 1), ("N", 0, 1)])
    norm8 = dict(M=4, N=512, group=48, x=MB, r=2 * MB, w=3 * MB, eps=1e-6, ro=4 * MB, out=5 * MB, sc=6 * MB, stream=0)
    tries("rglru_add_rmsnorm_e4m3", norm8, [("M", 0, 1), ("eps", -1.0, 1)])
    w4 = dict(M=65, N=100, K=256, group=64, A=MB, As=0, ag=0, W=2 * MB, Ws=3 * MB, b=4 * MB, out=5 * MB, stream=0)
    tries("rglru_linear_w4", w4, [("N", 0, 1), ("K", 0, 1)])
    at = {n: 16 * MB * (i + 1) for i, n in enumerate(NAMES)}
    sizes = dict(rows=8, S=2, H=4, Hkv=2, D=128, page=16, pages=8, max_pages=4, max_new=4, max_total=64)
    good_status = api.ERR_WORKSPACE
    append = dict(**sizes, **{n: at[n] for n in ("qkv", "cu", "ctx", "table")}, base=10000.0,
                  **{n: at[n] for n in ("q", "k", "ks", "v", "vs", "ws")}, wsb=16, stream=0)
    bad = [("rows", 0, 1), ("D", 64, 2), ("page", 24, 2), ("max_total", 65, 1), ("cu", 8, 1), ("table", 0, 1), ("vs", 8, 1),
           ("k", 8, 1), ("ws", 0, 3)]
    tries("rglru_paged_append", append, bad + [("wsb", 15, 3)])
    attend = dict(**sizes, window=32, scale=0.1, **{n: at[n] for n in ("qkv", "cu", "ctx", "table", "k", "ks", "v", "vs")},
                  out=at["q"], ws=at["ws"], wsb=16, stream=0)
    tries("rglru_paged_attention", attend, bad)
    good_status = api.ERR_INVALID_ARG
    room = dict(wsb=1 << 26)
    tries("rglru_paged_append", {**append, **room, "base": 1.0}, [("wsb", 16, 3)])
    tries("rglru_paged_append", {**append, **room, "q": 8}, [("wsb", 16, 3)])
    tries("rglru_paged_attention", {**attend, **room, "window": 0}, [("wsb", 16, 3)])
    tries("rglru_paged_attention", {**attend, **room, "scale": 0.0}, [("wsb", 16, 3)])
    tries("rglru_paged_attention", {**attend, **room, "out": at["v"]}, [("wsb", 16, 3)])
