"""The serving operators' C entry points and their binding on the CPU: argument
checks come before any HIP call, workspaces are planned without a device, and
the binding refuses what it should.  Nothing here launches a kernel."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from software_pipelined_tiled_pipeline_amd import fused, pgemm, serve  # noqa: E402

OK, NULL, SHAPE, ALIGN = 0, 1, 2, 4
A = 4096  # a pointer that is aligned and never read
BAD = A + 8
TYPES = ["f16", "bf16"]


@pytest.fixture(scope="module")
def L():
    return pgemm.lib()


def refusals(L, fmt, op, good, shapes, null, align):
    def call(**kw):
        return getattr(L, f"pgemm_{fmt}_{op}")(*{**good, **kw}.values())
    for kw in shapes:
        assert call(**kw) == SHAPE, kw
    for name in null:
        assert call(**{name: None}) == NULL, name
    for name in align:
        assert call(**{name: BAD}) == ALIGN, name
    return call


@pytest.mark.parametrize("fmt", TYPES)
def test_quant(L, fmt):
    good = dict(x=A, q=A, scale=A, M=8, K=8, stream=None)
    call = refusals(L, fmt, "quant_i8", good, [dict(M=-1), dict(K=-1), dict(M=(1 << 31) - 255), dict(K=(1 << 22) + 1)],
                    ["x", "q", "scale"], ["x", "q", "scale"])
    assert call(M=0, x=None, q=None, scale=None) == OK


@pytest.mark.parametrize("fmt", TYPES)
@pytest.mark.parametrize("gated", [False, True])
def test_i8(L, fmt, gated):
    good = dict(x=A, xs=A, w=A, ws=A, out=A, M=8, N=8, K=8)
    good.update(dict(act=0, stream=None) if gated else dict(stream=None))
    op = "i8_gated" if gated else "i8"
    # the largest K whose sums are exact: 128 * 128 * (2^17 - 16) is below 2^31
    assert 128 * 128 * ((1 << 17) - 16) < 1 << 31 <= 128 * 128 * (1 << 17)
    shapes = [dict(M=-1), dict(N=-1), dict(K=-1), dict(K=(1 << 17) - 15), dict(M=(1 << 31) - 255), dict(N=1 << 31),
              dict(M=1 << 30, N=1 << 12), dict(N=1 << 28)]
    call = refusals(L, fmt, op, good, shapes + ([dict(act=2)] if gated else []), ["x", "w", "ws", "out"],
                    ["x", "xs", "w", "ws", "out"])
    assert call(M=0, x=None, xs=None, out=None) == OK
    assert call(N=0, w=None, ws=None, out=None) == OK


@pytest.mark.parametrize("fmt", TYPES)
def test_moe(L, fmt):
    good = dict(x=A, router=A, w=A, down=A, y=A, experts=None, weights=None, M=8, E=8, D=8, F=8, k=2, normalize=1, act=0, stream=None)
    shapes = [dict(M=-1), dict(M=1 << 15), dict(E=0), dict(E=1025), dict(D=-1), dict(D=(1 << 22) + 1), dict(F=-1),
              dict(F=(1 << 17) + 1), dict(k=0), dict(k=9), dict(E=64, k=33), dict(act=2), dict(act=-1), dict(normalize=2)]
    call = refusals(L, fmt, "moe", good, shapes, ["x", "router", "w", "down", "y"],
                    ["x", "router", "w", "down", "y", "experts", "weights"])
    assert call(M=0, x=None, y=None) == OK


@pytest.mark.parametrize("fmt", TYPES)
def test_sample(L, fmt):
    good = dict(z=A, u=A, t=A, k=A, p=A, q=A, shared=0, token=A, M=8, V=8, stream=None)
    call = refusals(L, fmt, "sample", good, [dict(M=-1), dict(V=-1), dict(V=(1 << 30) + 1), dict(shared=16), dict(shared=-1)],
                    ["z", "u", "token"], ["z", "token"])
    for name in ("u", "t", "k", "p", "q"):  # single values: 4 bytes
        assert call(**{name: A + 2}) == ALIGN, name
    assert call(M=0, z=None, u=None, token=None) == OK


def test_workspaces(L):
    n = ctypes.c_int64(-1)
    assert L.pgemm_i8_workspace(8, 8, 8, 0, 0, None) == NULL and L.pgemm_moe_workspace(8, 8, 8, 8, 1, None) == NULL
    assert L.pgemm_i8_workspace(8, 8, -1, 0, 0, ctypes.byref(n)) == SHAPE
    assert L.pgemm_i8_workspace(8, 8, 1 << 17, 0, 0, ctypes.byref(n)) == SHAPE
    assert L.pgemm_moe_workspace(8, 8, 8, 8, 9, ctypes.byref(n)) == SHAPE
    assert L.pgemm_moe_workspace(1 << 15, 8, 8, 8, 1, ctypes.byref(n)) == SHAPE
    i8, moe = serve.i8_workspace_bytes, serve.moe_workspace_bytes
    # few tokens need none: their integers are given, or each workgroup makes them
    assert i8(8, 8192, 4096, False, True) == 0 and i8(2, 8192, 4096, False, False) == 0
    # else the tokens' integers and scales
    assert i8(2048, 8192, 4000, True, False) == 2048 * 4000 + 2048 * 4
    assert i8(2048, 8192, 4000, True, True) == 0
    # sums of pieces of K
    assert i8(300, 128, 16384, False, True) % (300 * 128 * 4) < 256 <= i8(300, 128, 16384, False, True)
    # logits, choices, weights, hidden values, their largest, products
    parts = [37 * 60 * 8, 37 * 4 * 4, 37 * 4 * 4, 37 * 4 * 1001 * 4, 37 * 4 * 4, 37 * 4 * 2050 * 4]
    assert moe(37, 60, 2050, 1001, 4) == sum(-(-p // 256) * 256 for p in parts)
    assert moe(0, 60, 2050, 1001, 4) == 0
    # nothing kept of one choice's products: they are the result
    assert moe(37, 60, 2050, 1001, 1) < 37 * 2050 * 4 + 37 * 1001 * 4


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 16, dtype=torch.float16), torch.zeros(4, 16, dtype=torch.int8)
    s, u = torch.zeros(4), torch.zeros(2)
    r, e, d = torch.zeros(3, 16).half(), torch.zeros(3, 8, 16).half(), torch.zeros(3, 16, 4).half()
    calls = [lambda: pgemm.pgemm_f16_quant_i8(x), lambda: pgemm.pgemm_f16_i8(x, w, s),
             lambda: pgemm.pgemm_f16_i8(w[:2], w, s, xs=u), lambda: pgemm.pgemm_f16_i8_gated(x, w, s),
             lambda: pgemm.pgemm_f16_moe(x, r, e, d, 2), lambda: pgemm.pgemm_f16_sample(x, u)]
    for c in calls:
        with pytest.raises(ValueError):
            c()


@pytest.mark.parametrize("fmt", TYPES)
@pytest.mark.parametrize("k", [0, -1, 33, 1 << 40, (1 << 64) + 1, -(1 << 64) + 2])
def test_top_k_of_a_mixture(fmt, k):
    # 2^64 + 1 would reach the library as 1
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError, match="top_k"):
        getattr(pgemm, f"pgemm_{fmt}_moe")(x, x, x, x, k)


@pytest.mark.parametrize("fmt", TYPES)
def test_act(fmt):
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError, match="act"):
        getattr(pgemm, f"pgemm_{fmt}_moe")(x, x, x, x, 1, act="relu")
    with pytest.raises(ValueError, match="act"):
        getattr(pgemm, f"pgemm_{fmt}_i8_gated")(x, x, x, act="tanh")


def test_functions_are_documented():
    assert not set(serve.SERVE_SYMBOLS) & set(fused.FUSED_SYMBOLS)
    for name in serve.SERVE_SYMBOLS:
        f = getattr(pgemm, name)
        assert f.__name__ == name and name in f.__doc__
