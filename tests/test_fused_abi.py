"""The fused operators' C entry points and their binding on the CPU: argument
checks come before any HIP call, workspaces are planned without a device, and
the binding refuses what it should.  Nothing here launches a kernel."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from software_pipelined_tiled_pipeline_amd import fused, pgemm  # noqa: E402

OK, NULL, SHAPE, ALIGN = 0, 1, 2, 4
A = 4096  # a pointer that is aligned and never read
BAD = A + 8
TYPES = ["f16", "bf16"]


@pytest.fixture(scope="module")
def L():
    return pgemm.lib()


def call(L, fmt, op, *args):
    return getattr(L, f"pgemm_{fmt}_{op}")(*args)


@pytest.mark.parametrize("fmt", TYPES)
def test_gated_refusals(L, fmt):
    good = dict(x=A, w=A, h=A, saved=None, M=8, F=8, D=8, act=0, stream=None)

    def gated(**kw):
        return call(L, fmt, "gated", *{**good, **kw}.values())
    for kw in (dict(M=-1), dict(F=-1), dict(D=-1), dict(M=1 << 31), dict(F=(1 << 21) + 1), dict(D=(1 << 22) + 1),
               dict(act=2), dict(act=-1), dict(M=(1 << 31) - 1, F=1 << 21, D=8)):
        assert gated(**kw) == SHAPE, kw
    for name in ("x", "w", "h"):
        assert gated(**{name: None}) == NULL, name
        assert gated(**{name: BAD}) == ALIGN, name
    assert gated(saved=BAD) == ALIGN
    # nothing to do: no device is asked for
    assert gated(M=0, x=None, h=None) == OK
    assert gated(F=0, w=None, h=None) == OK


@pytest.mark.parametrize("fmt", TYPES)
def test_gated_bwd_refusals(L, fmt):
    good = dict(dh=A, x=A, w=A, saved=None, dx=A, dw=A, M=8, F=8, D=8, act=1, stream=None)

    def bwd(**kw):
        return call(L, fmt, "gated_bwd", *{**good, **kw}.values())
    for kw in (dict(M=-1), dict(F=-2), dict(D=-1), dict(act=7), dict(F=1 << 22)):
        assert bwd(**kw) == SHAPE, kw
    for name in ("dh", "x", "w", "dx", "dw"):
        assert bwd(**{name: None}) == NULL, name
        assert bwd(**{name: BAD}) == ALIGN, name
    assert bwd(saved=BAD) == ALIGN
    assert bwd(D=0, x=None, w=None, dx=None, dw=None) == OK
    assert bwd(M=0, F=0, dh=None, x=None, w=None, dx=None, dw=None) == OK


@pytest.mark.parametrize("fmt", TYPES)
def test_xent_refusals(L, fmt):
    good = dict(x=A, w=A, target=A, loss=A, lse=A, M=8, V=8, D=8, ignore=-100, stream=None)

    def xent(**kw):
        return call(L, fmt, "xent", *{**good, **kw}.values())
    for kw in (dict(M=-1), dict(V=-1), dict(V=0), dict(D=-1), dict(D=(1 << 22) + 1), dict(V=1 << 31)):
        assert xent(**kw) == SHAPE, kw
    for name in ("x", "w", "target", "loss", "lse"):
        assert xent(**{name: None}) == NULL, name
        assert xent(**{name: BAD}) == ALIGN, name
    assert xent(M=0, x=None, target=None, loss=None, lse=None) == OK
    good = dict(dloss=A, step=1, x=A, w=A, target=A, lse=A, dx=A, dw=A, M=8, V=8, D=8, ignore=-100, stream=None)

    def bwd(**kw):
        return call(L, fmt, "xent_bwd", *{**good, **kw}.values())
    for kw in (dict(M=-1), dict(V=0), dict(D=-1), dict(step=2), dict(step=-1)):
        assert bwd(**kw) == SHAPE, kw
    for name in ("dloss", "x", "w", "target", "lse", "dx", "dw"):
        assert bwd(**{name: None}) == NULL, name
        if name != "dloss":
            assert bwd(**{name: BAD}) == ALIGN, name
    assert bwd(dloss=A + 2) == ALIGN
    assert bwd(D=0, x=None, w=None, dx=None, dw=None) == OK


@pytest.mark.parametrize("fmt", TYPES)
@pytest.mark.parametrize("gated", [False, True])
def test_q4_refusals(L, fmt, gated):
    good = dict(x=A, q=A, scale=A, zero=None, out=A, M=1, N=8, K=64, group=64)
    end = dict(act=0, stream=None) if gated else dict(stream=None)

    def q4(**kw):
        return call(L, fmt, "q4_gated" if gated else "q4", *{**good, **end, **kw}.values())
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(group=0), dict(group=-32), dict(group=48), dict(group=1 << 31),
               dict(K=(1 << 22) + 1), dict(M=(1 << 20)), dict(N=1 << 30, M=1)):
        # 2^30 output columns are too many for the gated block's 2^31 weight rows alone
        if kw == dict(N=1 << 30, M=1) and not gated:
            continue
        assert q4(**kw) == SHAPE, kw
    if gated:
        assert q4(act=2) == SHAPE
    for name in ("x", "q", "scale", "out"):
        assert q4(**{name: None}) == NULL, name
        assert q4(**{name: BAD}) == ALIGN, name
    assert q4(zero=BAD) == ALIGN
    assert q4(M=0, x=None, out=None) == OK
    assert q4(N=0, q=None, scale=None, out=None) == OK


def test_workspaces(L):
    n = ctypes.c_int64(-1)
    assert L.pgemm_fused_workspace(0, 8, 8, 8, None) == NULL
    for op, sizes in ((5, (8, 8, 8)), (-1, (8, 8, 8)), (0, (-1, 8, 8)), (3, (8, 0, 8)), (2, (8, 1 << 22, 8))):
        assert L.pgemm_fused_workspace(op, *sizes, ctypes.byref(n)) == SHAPE, (op, sizes)
    ws = fused.workspace_bytes
    # few rows, and rows that start on 16 bytes, need nothing
    assert ws("gated", 16, 12288, 4097) == 0
    assert ws("gated", 2048, 8192, 4096) == 0
    # odd rows: padded copies of both operands
    assert ws("gated", 300, 100, 1001) == 300 * 1008 * 2 + 128 + 200 * 1008 * 2  # parts on 256 bytes
    # the derivative by the projections
    assert ws("gated_bwd", 8192, 12288, 4096) == 8192 * 24576 * 2
    # statistics of every tile; at most 512 MiB of the derivative by the logits, and the running sum
    assert ws("xent", 8192, 65536, 4096) == 8192 * 512 * 8 + 8192 * 4
    big = ws("xent_bwd", 8192, 65536, 4096)
    assert (512 << 20) + 8192 * 4096 * 4 <= big <= (513 << 20) + 8192 * 4096 * 4
    for op in fused.FUSED_OPS:
        assert ws(op, 0, 5, 5) >= 0


def test_no_piece_of_the_vocabulary_is_short(L):
    # pieces are alike: the workspace for one more row of the vocabulary than
    # fits a piece is that of two halves
    one, two = fused.workspace_bytes("xent_bwd", 8192, 32768, 256), fused.workspace_bytes("xent_bwd", 8192, 32769, 256)
    assert two < one


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 8, dtype=torch.float16), torch.zeros(4, 8, dtype=torch.float16)
    t, f = torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    q, s = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.float16)
    calls = [lambda: pgemm.pgemm_f16_gated(x, w), lambda: pgemm.pgemm_f16_gated_bwd(x, x, w),
             lambda: pgemm.pgemm_f16_xent(x, w, t), lambda: pgemm.pgemm_f16_xent_bwd(f, x, w, t, f),
             lambda: pgemm.pgemm_f16_q4(x, q, s), lambda: pgemm.pgemm_f16_q4_gated(x, q, s)]
    for c in calls:
        with pytest.raises(ValueError):
            c()


def test_pack_q4():
    gen = torch.Generator().manual_seed(3)
    for n, k in ((1, 1), (3, 31), (2, 32), (5, 100)):
        v = torch.randint(0, 16, (n, k), generator=gen, dtype=torch.uint8)
        p = pgemm.pack_q4(v)
        assert p.shape == (n, -(-k // 32) * 16) and p.dtype == torch.uint8 and p.is_contiguous()
        back = torch.stack([p & 15, p >> 4], dim=2).reshape(n, -1)
        assert torch.equal(back[:, :k], v) and not back[:, k:].any()
    for bad in (torch.zeros(4, dtype=torch.uint8), torch.zeros(2, 2), torch.full((1, 1), 16, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            pgemm.pack_q4(bad)


def test_functions_are_documented():
    for name in fused.FUSED_SYMBOLS:
        f = getattr(pgemm, name)
        assert f.__name__ == name and name.rsplit("_", 1)[0][:9] in f.__doc__
