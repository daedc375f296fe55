"""The fused operators where they can go wrong: empty and masked input, values
past a type's range, long rows, offsets past 32 bits, streams, graphs,
workspaces and refusals.  Bounds as in tests/fused_reference.py."""
import ctypes
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fused_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, block, call, check, head, pg, q4_case, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu
FMT = ["f16", "bf16"]


def check_range(what, got, value, bound):
    """check(), where values may lie past the type's range: those come out infinite."""
    top = torch.finfo(got.dtype).max
    inside = value.abs() + bound < top
    check(what, got[inside], (value[inside], bound[inside]))
    past = value.abs() - bound > top * (1 + torch.finfo(got.dtype).eps)
    assert (got[past].double() == torch.sign(value[past]) * math.inf).all()


# ------------------------------------------------------------------ refusals

def test_refusals(pg):
    x, w, dh = block(1, "f16", 70, 40, 64)
    t = torch.zeros(70, dtype=torch.int64, device="cuda")
    f = torch.zeros(70, device="cuda")
    q, s = torch.zeros(80, 32, dtype=torch.uint8, device="cuda"), torch.zeros(80, 1, dtype=torch.float16, device="cuda")
    bad = [
        lambda: pg.pgemm_bf16_gated(x, w),                                        # type
        lambda: pg.pgemm_f16_gated(x.cpu(), w),                                   # device
        lambda: pg.pgemm_f16_gated(x, w[:, :32]),                                 # width, and not contiguous
        lambda: pg.pgemm_f16_gated(x, w[:79]),                                    # an odd number of rows
        lambda: pg.pgemm_f16_gated(x[0], w),                                      # one dimension
        lambda: pg.pgemm_f16_gated(x.t().contiguous().t(), w),                    # strides
        lambda: pg.pgemm_f16_gated(x, w, act="relu"),
        lambda: pg.pgemm_f16_gated(x, w, out=dh[:69]),
        lambda: pg.pgemm_f16_gated_bwd(dh[:, :39], x, w),
        lambda: pg.pgemm_f16_gated_bwd(dh, x, w, saved=f),
        lambda: pg.pgemm_f16_xent(x, w, t.int()),
        lambda: pg.pgemm_f16_xent(x, w, t[:69]),
        lambda: pg.pgemm_f16_xent_bwd(f.half(), x, w, t, f),
        lambda: pg.pgemm_f16_xent_bwd(f[:69], x, w, t, f),
        lambda: pg.pgemm_f16_xent_bwd(torch.zeros(140, device="cuda")[::2], x, w, t, f),
        lambda: pg.pgemm_f16_q4(x, q, s, group=48),
        lambda: pg.pgemm_f16_q4(x, q[:, :16], s, group=64),
        lambda: pg.pgemm_f16_q4(x, q, s.bfloat16(), group=64),
        lambda: pg.pgemm_f16_q4(x, q, s, zero=s, group=64),
        lambda: pg.pgemm_f16_q4_gated(x, q[:79], s[:79], group=64),
    ]
    for i, c in enumerate(bad):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"call {i} was not refused")
    # rows that start between two pieces of 16 bytes: the library's own refusal
    odd = torch.zeros(71 * 63, dtype=torch.float16, device="cuda")[63:].view(70, 63)
    with pytest.raises(pg.PgemmError) as e:
        pg.pgemm_f16_gated(odd, w[:, :63].contiguous())
    assert e.value.status == 4


def test_workspace_that_is_missing_or_too_small(pg):
    # nothing is enqueued: the outputs keep what they held
    stream = torch.cuda.Stream()
    M, V, D = 70, 300, 64
    x, w, target, _ = head(2, "f16", M, V, D)
    loss, lse = torch.full((M,), 7.0, device="cuda"), torch.full((M,), 7.0, device="cuda")
    need = pg.fused.workspace_bytes("xent", M, V, D)
    room = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    L, h = pg.lib(), ctypes.c_void_p(stream.cuda_stream)

    def xent():
        return L.pgemm_f16_xent(x.data_ptr(), w.data_ptr(), target.data_ptr(), loss.data_ptr(), lse.data_ptr(), M, V, D,
                                -100, h)
    assert xent() == 9
    assert L.pgemm_set_workspace(h, room.data_ptr(), need - 1) == 0
    assert xent() == 9
    torch.cuda.synchronize()
    assert (loss == 7).all() and (lse == 7).all()
    assert L.pgemm_set_workspace(h, room.data_ptr(), need) == 0
    assert xent() == 0
    torch.cuda.synchronize()
    check("lse", lse, ref.xent(x, w, target)["lse"])
    assert L.pgemm_set_workspace(h, None, 0) == 0


@pytest.mark.parametrize("fmt", FMT)
def test_outputs_of_the_callers_own(pg, fmt):
    # the same values, in the tensors that were given
    def same(name, args, kw, **outs):
        got = call(pg, fmt, name, *args, **kw, **outs)
        want = call(pg, fmt, name, *args, **kw)
        got, want = (t if isinstance(t, tuple) else (t,) for t in (got, want))
        for g, w, o in zip(got, want, outs.values()):
            assert g is o and torch.equal(g, w)

    def like(*shape, dtype=TYPES[fmt]):
        return torch.full(shape, math.nan, dtype=dtype, device="cuda")
    M, F, D, V = 90, 40, 72, 333
    x, w, dh = block(23, fmt, M, F, D)
    same("gated", (x, w), dict(act="gelu"), out=like(M, F))
    _, saved = call(pg, fmt, "gated", x, w, save=True)
    same("gated_bwd", (dh, x, w), dict(saved=saved), dx=like(M, D), dw=like(2 * F, D))
    hx, hw, target, dloss = head(24, fmt, M, V, D)
    same("xent", (hx, hw, target), {}, loss=like(M, dtype=torch.float32), lse=like(M, dtype=torch.float32))
    _, lse = call(pg, fmt, "xent", hx, hw, target)
    same("xent_bwd", (dloss, hx, hw, target, lse), {}, dx=like(M, D), dw=like(V, D))
    tok, values, scale, zero = q4_case(25, fmt, 3, 64, 200, 64, True)
    packed = pg.pack_q4(values)
    same("q4", (tok, packed, scale, zero), dict(group=64), out=like(3, 64))
    same("q4_gated", (tok, packed, scale, zero), dict(group=64, act="gelu"), out=like(3, 32))


# ------------------------------------------------------------ empty and masked

@pytest.mark.parametrize("fmt", FMT)
def test_empty(pg, fmt):
    for M, F, D in ((0, 5, 8), (5, 0, 8), (70, 6, 0), (0, 0, 8), (0, 5, 0)):
        x, w, dh = block(3, fmt, M, F, D)
        h, saved = call(pg, fmt, "gated", x, w, save=True)
        assert h.shape == (M, F) and not h.any()
        assert not call(pg, fmt, "gated", x, w).any()
        for keep in (saved, None):
            dx, dw = call(pg, fmt, "gated_bwd", dh, x, w, saved=keep)
            assert dx.shape == (M, D) and dw.shape == (2 * F, D) and not dx.any() and not dw.any()
    for M, V, D in ((0, 300, 8), (70, 300, 0), (0, 3, 0)):
        x, w, target, dloss = head(4, fmt, M, V, max(D, 1))
        x, w = x[:, :D].contiguous(), w[:, :D].contiguous()
        loss, lse = call(pg, fmt, "xent", x, w, target)
        if M:  # all logits are zero
            assert torch.allclose(lse, torch.full_like(lse, math.log(V)), rtol=1e-6)
        dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, target, lse)
        assert dx.shape == (M, D) and dw.shape == (V, D) and not dx.any() and not dw.any()
    for M, N, K in ((0, 5, 64), (3, 0, 64), (3, 6, 0)):
        x, values, scale, zero = q4_case(5, fmt, M, N, K, 64, True)
        assert not call(pg, fmt, "q4", x, pg.pack_q4(values), scale, zero, group=64).any()
        if N % 2 == 0:
            assert not call(pg, fmt, "q4_gated", x, pg.pack_q4(values), scale, zero, group=64).any()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,V,D", [(3, 70, 40), (300, 5000, 72)])
def test_ignored_rows(pg, fmt, M, V, D):
    x, w, target, dloss = head(6, fmt, M, V, D)
    # no row counts
    none = torch.full_like(target, -100)
    loss, lse = call(pg, fmt, "xent", x, w, none)
    assert not loss.any()
    check("lse", lse, ref.xent(x, w, none)["lse"])
    dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, none, lse)
    assert not dx.any() and not dw.any()
    # one does, and any value may stand for those that do not, inside the vocabulary or not
    for ignore in (-100, -1, 5, V + 3):
        one = torch.full_like(target, ignore)
        one[M // 2] = V - 1
        want = ref.xent(x, w, one, ignore=ignore, dloss=dloss)
        loss, lse = call(pg, fmt, "xent", x, w, one, ignore_index=ignore)
        check("loss", loss, want["loss"])
        dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, one, lse, ignore_index=ignore)
        check("dx", dx, want["dx"])
        check("dw", dw, want["dw"])
    # what an ignored row holds does not matter to its loss and dx
    one = torch.full_like(target, -100)
    one[0] = 1
    for poison in (math.nan, math.inf, -math.inf, torch.finfo(x.dtype).min, torch.finfo(x.dtype).max):
        y = x.clone()
        y[1:] = poison
        loss, lse = call(pg, fmt, "xent", y, w, one)
        assert not loss[1:].any()
        dx, _ = call(pg, fmt, "xent_bwd", dloss, y, w, one, lse)
        assert not dx[1:].any() and dx[0].isfinite().all() and dx[0].any()


@pytest.mark.parametrize("fmt", FMT)
def test_targets_outside_the_vocabulary(pg, fmt):
    M, V, D = 130, 500, 64
    x, w, target, dloss = head(7, fmt, M, V, D)
    for wrong in (-1, V, 1 << 40, -(1 << 40)):
        t = target.clone()
        t[17] = wrong
        loss, lse = call(pg, fmt, "xent", x, w, t)
        assert loss[17].isnan() and loss.isnan().sum() == 1 and lse.isfinite().all()
        dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, t, lse)
        assert dx[17].isnan().all() and not dx[:17].isnan().any() and not dx[18:].isnan().any()
        assert dw.isnan().all()


@pytest.mark.parametrize("fmt", FMT)
def test_weights_of_the_loss(pg, fmt):
    M, V, D = 140, 900, 64
    x, w, target, _ = head(8, fmt, M, V, D)
    _, lse = call(pg, fmt, "xent", x, w, target)
    one = torch.full((1,), 0.37, device="cuda")
    want = ref.xent(x, w, target, dloss=one)
    for dloss in (one[0], one.expand(M), one.expand(M).contiguous()):
        dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, target, lse)
        check("dx", dx, want["dx"])
        check("dw", dw, want["dw"])
    gen = torch.Generator().manual_seed(9)
    mixed = randn(gen, M).cuda()
    mixed[::3] = 0
    for scale in (1e-3, 1.0, 300.0):  # of both signs, some of them zero
        want = ref.xent(x, w, target, dloss=mixed * scale)
        dx, dw = call(pg, fmt, "xent_bwd", mixed * scale, x, w, target, lse)
        check("dx", dx, want["dx"])
        check("dw", dw, want["dw"])
    dx, dw = call(pg, fmt, "xent_bwd", mixed * 0, x, w, target, lse)
    assert not dx.any() and not dw.any()


# ------------------------------------------------------------------ values

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [3, 200])
def test_gate_far_from_zero(pg, fmt, act, M):
    # projections that are single products: gates to either side of where the
    # activation is flat, and h past the type's range
    D = F = 64
    x = torch.zeros(M, D, dtype=TYPES[fmt], device="cuda")
    steps = torch.tensor([0.0, 1e-4, 0.3, 1.0, 4.0, 9.0, 12.0, 40.0, 100.0, 1000.0, 60000.0], device="cuda")
    values = torch.cat([steps, -steps]).to(x.dtype)
    x[:, 0] = values[torch.arange(M, device="cuda") % len(values)]
    x[:, 1] = 1
    w = torch.zeros(2 * F, D, dtype=x.dtype, device="cuda")
    w[:F, 0] = 1
    w[F:, 1] = torch.linspace(-3, 3, F, device="cuda").to(x.dtype)
    dh = torch.full((M, F), 0.5, dtype=x.dtype, device="cuda")
    want = ref.gated(x, w, act, dh)
    h, saved = call(pg, fmt, "gated", x, w, act=act, save=True)
    for got in (h, call(pg, fmt, "gated", x, w, act=act)):
        check_range("h", got, *want["h"])
    for keep in (saved, None):
        dx, dw = call(pg, fmt, "gated_bwd", dh, x, w, saved=keep, act=act)
        check_range("dx", dx, *want["dx"])
        check_range("dw", dw[:, 1], *(v[:, 1] for v in want["dw"]))
        assert not dx.isnan().any() and not dw.isnan().any()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [2, 150])
def test_nan_stays_where_it_belongs(pg, fmt, M):
    x, w, dh = block(10, fmt, M, 40, 72)
    x[1, 3] = math.nan
    h, saved = call(pg, fmt, "gated", x, w, save=True)
    for got in (h, call(pg, fmt, "gated", x, w)):
        assert got[1].isnan().all() and not got[0].isnan().any() and not got[2:].isnan().any()
    dx, dw = call(pg, fmt, "gated_bwd", dh, x, w, saved=saved)
    assert dx[1].isnan().all() and not dx[0].isnan().any() and dw.isnan().all()
    x, w, target, dloss = head(11, fmt, M, 400, 72)
    target[:] = 3
    w[7, 1] = math.nan  # a vocabulary row: every row's softmax
    loss, lse = call(pg, fmt, "xent", x, w, target)
    assert loss.isnan().all() and lse.isnan().all()
    x, values, scale, zero = q4_case(12, fmt, M, 50, 200, 64, True)
    scale[9, 1] = math.nan
    y = call(pg, fmt, "q4", x, pg.pack_q4(values), scale, zero, group=64)
    assert y[:, 9].isnan().all() and not y[:, :9].isnan().any() and not y[:, 10:].isnan().any()


@pytest.mark.parametrize("fmt", FMT)
def test_logits_far_apart(pg, fmt):
    # one logit that takes all of the softmax, rows whose logits are all alike,
    # and logits whose exponentials leave fp32 without their maximum taken off
    M, V, D = 130, 1000, 64
    x = torch.zeros(M, D, dtype=TYPES[fmt], device="cuda")
    w = torch.zeros(V, D, dtype=TYPES[fmt], device="cuda")
    w[:, 0] = torch.linspace(-200, 200, V, device="cuda").to(w.dtype)
    x[:, 0] = torch.linspace(-30, 30, M, device="cuda").to(x.dtype)
    x[5] = 0
    target = torch.arange(M, device="cuda") * 7 % V
    dloss = torch.ones(M, device="cuda")
    want = ref.xent(x, w, target, dloss=dloss)
    loss, lse = call(pg, fmt, "xent", x, w, target)
    check("lse", lse, want["lse"])
    check("loss", loss, want["loss"])
    dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, target, lse)
    check("dx", dx, want["dx"])
    check("dw", dw, want["dw"])


# ------------------------------------------------------------------- sizes

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,F,D", [(40, 6000, 104), (129, 5000, 260), (600, 100, 1024), (520, 2000, 72)])
def test_gated_in_pieces_of_k(pg, fmt, M, F, D):
    x, w, dh = block(13, fmt, M, F, D)
    want = ref.gated(x, w, "silu", dh)
    _, saved = call(pg, fmt, "gated", x, w, save=True)
    first = call(pg, fmt, "gated_bwd", dh, x, w, saved=saved)
    check("dx", first[0], want["dx"])
    check("dw", first[1], want["dw"])
    again = call(pg, fmt, "gated_bwd", dh, x, w, saved=saved)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])  # summed in one order


# few tokens with a long vocabulary; pieces of the vocabulary whose dx is summed in pieces of K
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,V,D", [(75, 13120, 352), (2100, 130001, 72)])
def test_xent_in_pieces(pg, fmt, M, V, D):
    x, w, target, dloss = head(14, fmt, M, V, D)
    want = ref.xent(x, w, target, dloss=dloss)
    loss, lse = call(pg, fmt, "xent", x, w, target)
    check("lse", lse, want["lse"])
    check("loss", loss, want["loss"])
    dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, target, lse)
    check("dx", dx, want["dx"])
    check("dw", dw, want["dw"])


# every number of tokens a workgroup may hold by every kind of group, rows
# shorter than a fragment, more k than a workgroup keeps scales of, and as
# many weight rows as each arrangement of waves takes
Q4 = [(M, 70, K, group) for M in (1, 4, 5, 16, 20, 40, 64, 65) for K, group in
      ((3, 32), (40, 64), (128, 32), (1000, 128), (8200, 96), (20000, 64))] + [
    (1, 8190, 1100, 128), (1, 9000, 300, 64), (2, 16500, 700, 32), (9, 8200, 260, 128), (7, 9000, 390, 32),
    (20, 16400, 300, 64), (40, 16400, 200, 32), (64, 16500, 130, 128), (3, 40, 40000, 32), (33, 40, 40000, 16384)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K,group", Q4)
def test_q4_sizes(pg, fmt, M, N, K, group):
    x, values, scale, zero = q4_case(M + N + K, fmt, M, N, K, group, True)
    scale[::3] *= -1
    packed = pg.pack_q4(values)
    for z in (zero, None):
        check("y", call(pg, fmt, "q4", x, packed, scale, z, group=group), ref.q4(x, values, scale, z, group))
    check_range("h", call(pg, fmt, "q4_gated", x, packed, scale, zero, group=group, act="gelu"),
                *ref.q4(x, values, scale, zero, group, act="gelu"))


# two, three and four waves beside each other, 16 tokens a workgroup with more
# than 16 of them, more than one stretch of scales, and
# every number of blocks that a wave may be left with
Q4_WAVES = [(24, 16420, 4500, 32), (48, 16400, 1000, 64), (33, 16400, 2500, 96), (130, 8200, 700, 32),
            (50, 16390, 2200, 32), (24, 13000, 4500, 32), (40, 13010, 1000, 64), (60, 13020, 300, 128),
            (31, 130, 8300, 32), (64, 500, 1450, 64), (100, 2000, 520, 128)] + [(M, 48, 128 * blocks - 5, 32) for M in (3, 11, 30) for blocks in (5, 9, 18, 27, 37)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K,group", Q4_WAVES)
def test_q4_waves(pg, fmt, M, N, K, group):
    x, values, scale, zero = q4_case(M + N + K, fmt, M, N, K, group, True)
    packed = pg.pack_q4(values)
    check("y", call(pg, fmt, "q4", x, packed, scale, zero, group=group), ref.q4(x, values, scale, zero, group))
    check_range("h", call(pg, fmt, "q4_gated", x, packed, scale, zero, group=group, act="silu"),
                *ref.q4(x, values, scale, zero, group, act="silu"))


@pytest.mark.parametrize("fmt", FMT)
def test_q4_any_byte_as_zero_point(pg, fmt):
    x, values, scale, _ = q4_case(15, fmt, 5, 256, 256, 32, True)
    zero = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].expand(256, 8).contiguous()
    y = call(pg, fmt, "q4", x, pg.pack_q4(values), scale, zero, group=32)
    value, _ = ref.q4(x, values, scale, zero, 32)
    # sums of x (16 + q) and x (16 + zero), each at most 271 sum |x|
    size = 2 * 271 * (x.double().abs() @ scale.double()[:, torch.arange(256, device="cuda") // 32].abs().t())
    bound = (32 + 8 + 16) * ref.U32 * size
    check("y", y, (value, bound + ref.half_step(x.dtype) * (value.abs() + bound) + ref.tiny(x.dtype)))


def test_offsets_past_32_bits(pg):
    # h has 2.3e9 values, and the last rows are compared
    M, F, D = 1100, 1 << 21, 8
    gen = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(2 * F, D, generator=gen, device="cuda") * 0.4).bfloat16()
    h = pg.pgemm_bf16_gated(x, w)
    some = torch.cat([torch.arange(3), torch.randint(0, F, (500,)), torch.arange(F - 3, F)]).cuda()
    rows = torch.tensor([0, 1023, 1024, M - 1], device="cuda")
    want = ref.gated(x[rows], torch.cat([w[some], w[F + some]]), "silu")["h"]
    check("h", h[rows][:, some], want)


# ------------------------------------------------------- gradients by differences

def test_xent_gradient_by_differences(pg):
    # loss is fp32; x moves by e to either side, exactly in f16.  The central
    # difference is off by at most e^2 / 6 times the third derivative, which is
    # at most the cube of the logits' change per step of x, and by the two
    # losses' own errors over 2 e.
    M, V, D, e = 4, 300, 16, 2.0 ** -5
    gen = torch.Generator().manual_seed(17)
    x = (torch.randint(-64, 65, (M, D), generator=gen).float() / 32).half().cuda()
    w = randn(gen, V, D, scale=0.5).half().cuda()
    target = torch.randint(0, V, (M,), generator=gen).cuda()
    _, lse = pg.pgemm_f16_xent(x, w, target)
    dx, _ = pg.pgemm_f16_xent_bwd(torch.ones((), device="cuda"), x, w, target, lse)
    reach = (w.double().max(0).values - w.double().min(0).values) ** 3
    for d in range(D):
        up, down = x.clone(), x.clone()
        up[:, d] += e
        down[:, d] -= e
        slope = (pg.pgemm_f16_xent(up, w, target)[0].double() - pg.pgemm_f16_xent(down, w, target)[0].double()) / (2 * e)
        own = ref.xent(up, w, target)["loss"][1] + ref.xent(down, w, target)["loss"][1]
        rounding = ref.xent(x, w, target, dloss=torch.ones(1, device="cuda"))["dx"][1][:, d]
        check("dx", dx[:, d], (slope, e * e / 6 * reach[d] + own / (2 * e) + rounding))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_by_differences(pg, act):
    # the sum of dh h in 64 bits of the rounded h: the difference is off by the
    # two h's bounds over 2 e and by e^2 / 6 times the third derivative of
    # a(g) u along x, at most 3 in a's first three derivatives each
    M, F, D, e = 5, 24, 16, 0.125
    gen = torch.Generator().manual_seed(18)
    x = (torch.randint(-8, 9, (M, D), generator=gen).float() / 8).half().cuda()
    w = randn(gen, 2 * F, D, scale=0.25).half().cuda()
    dh = torch.ones(M, F, dtype=torch.float16, device="cuda")
    dx, _ = pg.pgemm_f16_gated_bwd(dh, x, w, act=act)
    want = ref.gated(x, w, act, dh)["dx"]
    wg, wu = w[:F].double(), w[F:].double()
    u = (x.double() @ wu.t()).abs().max()
    for d in range(D):
        up, down = x.clone(), x.clone()
        up[:, d] += e
        down[:, d] -= e
        a, b = pg.pgemm_f16_gated(up, w, act=act), pg.pgemm_f16_gated(down, w, act=act)
        slope = (a.double() - b.double()).sum(1) / (2 * e)
        own = (ref.gated(up, w, act)["h"][1] + ref.gated(down, w, act)["h"][1]).sum(1) / (2 * e)
        third = (3 * wg[:, d].abs() ** 3 * (u + e) + 3 * 3 * wg[:, d] ** 2 * wu[:, d].abs()).sum()
        check("dx", dx[:, d], (slope, own + e * e / 6 * third + want[1][:, d]))


# ------------------------------------------------------------ streams and graphs

@pytest.mark.parametrize("fmt", FMT)
def test_other_streams(pg, fmt):
    x, w, dh = block(19, fmt, 200, 90, 101)
    here, saved = call(pg, fmt, "gated", x, w, save=True)
    grads = call(pg, fmt, "gated_bwd", dh, x, w, saved=saved)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    h, s = call(pg, fmt, "gated", x, w, save=True, stream=stream)
    dx, dw = call(pg, fmt, "gated_bwd", dh, x, w, saved=s, stream=stream)
    with torch.cuda.stream(stream):
        again = call(pg, fmt, "gated_bwd", dh, x, w, saved=s)
    stream.synchronize()
    assert torch.equal(h, here)
    for got in ((dx, dw), again):
        assert torch.equal(got[0], grads[0]) and torch.equal(got[1], grads[1])
    pg.release_workspace(stream)


@pytest.mark.parametrize("fmt", FMT)
def test_graph(pg, fmt):
    # a training step and a token's product recorded together, replayed on
    # other inputs with eager calls of larger ones in between
    M, F, D, V = 150, 90, 101, 700
    x, w, dh = block(20, fmt, M, F, D)
    hx, head_w, target, dloss = head(21, fmt, M, V, D)
    tok, values, scale, zero = q4_case(22, fmt, 3, 64, 200, 64, True)
    packed = pg.pack_q4(values)

    def step():
        h, saved = call(pg, fmt, "gated", x, w, save=True)
        loss, lse = call(pg, fmt, "xent", x, head_w, target)
        return [h, *call(pg, fmt, "gated_bwd", dh, x, w, saved=saved), loss,
                *call(pg, fmt, "xent_bwd", dloss, x, head_w, target, lse),
                call(pg, fmt, "q4", tok, packed, scale, zero, group=64)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        gen = torch.Generator().manual_seed(30 + turn)
        x.copy_(randn(gen, M, D).to(x.dtype))
        tok.copy_(randn(gen, 3, 200).to(tok.dtype))
        target.copy_(torch.randint(0, V, (M,), generator=gen))
        want = [t.clone() for t in step()]
        # a larger call replaces the stream's workspace, and new tensors take its place
        big = block(40 + turn, fmt, 300 + 100 * turn, 210, 333)
        call(pg, fmt, "gated_bwd", big[2], big[0], big[1])
        junk = [torch.full((1 << 20,), math.nan, device="cuda") for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        del junk
    pg.release_workspace(side)
