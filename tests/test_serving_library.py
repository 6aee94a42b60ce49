"""The serving calls without a GPU: exported, and every bad argument refused
before anything touches CUDA; the binding refuses what is no CUDA tensor."""
import pytest
import torch

import verifiable_quantize_rows_gb300 as bsg
from verifiable_quantize_rows_gb300 import build, serving

D = 4096            # a dummy device address, 256-byte aligned, never read
ARG, WORKSPACE = 1, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bsg.load()


def test_declared():
    names = bsg.exported_symbols()
    for n in ("bsg_wquant_groups", "bsg_wgroups_matvec", "bsg_kv8_append", "bsg_kv8_attend",
              "bsg_kv8_attend_workspace_size", "bsg_logprobs", "bsg_logprobs_backward"):
        assert n in names


def refused(fn, good, changes, code=ARG):
    """Each change of one argument of a good call is refused with `code`."""
    args = list(good.values())
    assert fn(*args) not in (ARG, WORKSPACE)      # only the missing device is left to object to
    for name, value in changes:
        bad = dict(good, **{name: value})
        assert fn(*bad.values()) == code, (name, value)


def test_wquant_groups(lib):
    good = dict(W=D, K=100, N=7, ldw=7, group=32, Q=D, ldq=4, scale=D, lds=7, st=None, stream=None)
    refused(lib.bsg_wquant_groups, good,
            [("W", None), ("W", D + 1), ("Q", None), ("scale", None), ("scale", D + 2), ("K", 0), ("N", 0),
             ("K", 1 << 31), ("ldw", 6), ("ldq", 3), ("lds", 6), ("group", -32), ("group", 16), ("group", 33)])


def test_wgroups_matvec(lib):
    good = dict(X=D, dtype=0, ldx=100, Q=D, ldq=4, scale=D, lds=7, group=32, M=3, N=7, K=100, relu=0, Y=D, ldy=7,
                ws=D, n=lib.bsg_wgroups_matvec_workspace_size(3, 7, 100), st=None, stream=None)
    refused(lib.bsg_wgroups_matvec, good,
            [("X", None), ("X", D + 2), ("dtype", 3), ("dtype", -1), ("ldx", 99), ("Q", None), ("ldq", 3), ("scale", None),
             ("lds", 6), ("group", 48), ("M", 0), ("M", 17), ("N", 0), ("K", 0), ("relu", 2), ("Y", None), ("ldy", 6),
             ("N", (1 << 25) + 1), ("K", (1 << 30) + 1)])
    assert good["n"] == 0  # small products need none
    good.update(M=5, n=lib.bsg_wgroups_matvec_workspace_size(5, 7, 100))
    refused(lib.bsg_wgroups_matvec, good, [("ws", None), ("ws", D + 16), ("n", good["n"] - 1)], WORKSPACE)
    assert lib.bsg_wgroups_matvec_workspace_size(0, 5, 5) == lib.bsg_wgroups_matvec_workspace_size(17, 5, 5) == 0


def cache(**kw):
    c = dict(k=D, v=D, k_scale=D, v_scale=D, pages=10, heads=2, page_tokens=16, dim=64)
    return serving._CACHE.pack(*(0 if x is None else x for x in dict(c, **kw).values()))


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=D + 8), dict(v=D + 1), dict(k_scale=None), dict(v_scale=D + 2),
              dict(pages=0), dict(pages=1 << 31), dict(heads=0), dict(heads=65536), dict(page_tokens=8),
              dict(page_tokens=24), dict(page_tokens=1040), dict(dim=48), dict(dim=0), dict(dim=512)]


def tokens(data=D):
    return serving._TOKENS.pack(data or 0, 128, 128, 64)


def test_kv8_append(lib):
    good = dict(cache=cache(), table=D, ld=4, starts=D, counts=None, k=tokens(), v=tokens(), dtype=1, B=2, T=3, st=None,
                stream=None)
    refused(lib.bsg_kv8_append, good,
            [("cache", None), *[("cache", cache(**c)) for c in BAD_CACHES], ("table", None), ("table", D + 1), ("ld", 0),
             ("ld", 1 << 30), ("starts", None), ("k", None), ("v", None), ("k", tokens(None)), ("v", tokens(D + 1)),
             ("dtype", 5), ("B", 0), ("B", 65536), ("T", 0), ("T", 1 << 30)])


def test_kv8_attend(lib):
    size = lib.bsg_kv8_attend_workspace_size(cache(), 4, 2, 3, 4)
    assert size > 0
    for bad in BAD_CACHES:
        assert lib.bsg_kv8_attend_workspace_size(cache(**bad), 4, 2, 3, 4) == 0
    for bad in ((0, 2, 3, 4), (4, 0, 3, 4), (4, 2, 0, 4), (4, 2, 17, 4), (4, 2, 3, 3), (4, 2, 3, 0)):
        assert lib.bsg_kv8_attend_workspace_size(cache(), *bad) == 0
    good = dict(cache=cache(), table=D, ld=4, lens=D, q=tokens(), out=tokens(), dtype=0, B=2, T=3, heads=4, scale=0.1,
                lse=None, ws=D, n=size, st=None, stream=None)
    refused(lib.bsg_kv8_attend, good,
            [("cache", None), *[("cache", cache(**c)) for c in BAD_CACHES], ("table", None), ("ld", 0), ("lens", None),
             ("q", None), ("out", None), ("q", tokens(D + 2)), ("out", tokens(None)), ("dtype", 3), ("B", 0), ("T", 0),
             ("T", 17), ("heads", 3), ("heads", 0), ("heads", 1 << 17), ("scale", float("inf")), ("scale", float("nan"))])
    refused(lib.bsg_kv8_attend, good, [("ws", None), ("ws", D + 128), ("n", size - 1), ("n", 0)], WORKSPACE)


def test_logprobs(lib):
    good = dict(x=D, dtype=0, M=3, V=10, ldl=10, target=None, top=2, lp=None, ent=None, lse=None, tl=D, ti=D, st=None,
                stream=None)
    refused(lib.bsg_logprobs, good,
            [("x", None), ("x", D + 1), ("dtype", 9), ("M", 0), ("V", 0), ("V", 1 << 31), ("ldl", 9), ("top", -1), ("top", 33),
             ("top", 11), ("tl", None), ("ti", None)])
    good = dict(x=D, dtype=2, M=3, V=10, ldl=10, target=None, lse=D, ent=D, gl=None, gh=D, dx=D, ldd=10, st=None, stream=None)
    refused(lib.bsg_logprobs_backward, good,
            [("x", None), ("dtype", 3), ("M", 0), ("V", 0), ("ldl", 9), ("lse", None), ("ent", None), ("dx", None), ("dx", D + 1),
             ("ldd", 9), ("ldd", 11)])


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.ones(2, 64)
    for call in (lambda: bsg.wquant_groups(x), lambda: bsg.wgroups_matvec(x, x, x), lambda: bsg.logprobs(x),
                 lambda: bsg.logprobs_backward(x, None, x[0]),
                 lambda: bsg.kv8_append(x[None, None], x[None, None], (x, x, x, x), x, x),
                 lambda: bsg.kv8_attend(x[None, None], (x, x, x, x), x, x)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError, match="CUDA tensor"):
        bsg.logprobs(x.double())
    with pytest.raises(AttributeError):
        bsg.no_such_name
