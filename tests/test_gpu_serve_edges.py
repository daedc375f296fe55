"""The serving operators where they can go wrong: empty and masked input, ties,
infinities and NaN, values past a type's range, offsets past 32 bits, streams,
graphs, workspaces and refusals.  References and bounds as in
tests/serve_reference.py."""
import ctypes
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, call, check, pg, randn  # noqa: E402,F401
from test_gpu_fused_edges import check_range  # noqa: E402
from test_gpu_serve import check_moe, equal, i8_case, moe_case, on_gpu, settings  # noqa: E402

pytestmark = pytest.mark.gpu
FMT = ["f16", "bf16"]


# ------------------------------------------------------------------ refusals

def test_refusals(pg):
    x, w, s = i8_case(1, "f16", 6, 8, 50, False)
    q, xs = ref.quant(x)
    m = moe_case(2, "f16", 3, 16, 8, 4)
    z, u = torch.zeros(3, 50, dtype=torch.float16, device="cuda"), torch.zeros(3, device="cuda")
    one = torch.ones((), device="cuda")
    bad = [
        lambda: pg.pgemm_bf16_quant_i8(x),                                  # type
        lambda: pg.pgemm_f16_quant_i8(x.cpu()),                             # device
        lambda: pg.pgemm_f16_quant_i8(x.t()),                               # strides
        lambda: pg.pgemm_f16_quant_i8(x[0]),
        lambda: pg.pgemm_f16_quant_i8(x, q=q[:, :48]),
        lambda: pg.pgemm_f16_quant_i8(x, scale=xs.half()),
        lambda: pg.pgemm_f16_i8(x, w[:, :48].contiguous(), s),              # width
        lambda: pg.pgemm_f16_i8(x, w.view(torch.uint8), s),
        lambda: pg.pgemm_f16_i8(x, w, s[:7]),
        lambda: pg.pgemm_f16_i8(x, w, s.double()),
        lambda: pg.pgemm_f16_i8(q, w, s),                                   # integers without scales
        lambda: pg.pgemm_f16_i8(x, w, s, xs=xs),                            # scales without integers
        lambda: pg.pgemm_f16_i8(q, w, s, xs=xs[:5]),
        lambda: pg.pgemm_f16_i8(q[:, :50].contiguous(), w, s, xs=xs),       # rows that are no multiple of 16
        lambda: pg.pgemm_f16_i8(x, w, s, out=z),
        lambda: pg.pgemm_f16_i8_gated(x, w[:7], s[:7]),
        lambda: pg.pgemm_f16_i8_gated(x, w, s, act="relu"),
        lambda: pg.pgemm_bf16_moe(*m, 2),
        lambda: pg.pgemm_f16_moe(m[0], m[1][:3], m[2], m[3], 2),            # experts
        lambda: pg.pgemm_f16_moe(m[0], m[1], m[2][:, :15].contiguous(), m[3], 2),
        lambda: pg.pgemm_f16_moe(m[0], m[1], m[2], m[3][:, :, :7].contiguous(), 2),
        lambda: pg.pgemm_f16_moe(m[0], m[1], m[2].transpose(0, 1), m[3], 2),
        lambda: pg.pgemm_f16_moe(*m, 5),                                    # more than there are
        lambda: pg.pgemm_f16_moe(*m, 2, out=z),
        lambda: pg.pgemm_f16_sample(z, u[:2]),
        lambda: pg.pgemm_f16_sample(z, u.double()),
        lambda: pg.pgemm_f16_sample(z.float(), u),
        lambda: pg.pgemm_f16_sample(z, u, temperature=0.5),
        lambda: pg.pgemm_f16_sample(z, u, top_k=u),
        lambda: pg.pgemm_f16_sample(z, u, top_p=one.cpu()),
        lambda: pg.pgemm_f16_sample(z, u, min_p=one.expand(3)),
        lambda: pg.pgemm_f16_sample(z, u, token=torch.zeros(3, dtype=torch.int32, device="cuda")),
    ]
    for i, c in enumerate(bad):
        with pytest.raises((ValueError, AttributeError)):
            c()
            pytest.fail(f"call {i} was not refused")
    # rows that start between two pieces of 16 bytes: the library's own refusal
    odd = torch.zeros(7 * 50, dtype=torch.float16, device="cuda")[50:].view(6, 50)
    for c in (lambda: pg.pgemm_f16_quant_i8(odd), lambda: pg.pgemm_f16_i8(odd, w, s), lambda: pg.pgemm_f16_sample(odd[:3], u)):
        with pytest.raises(pg.PgemmError) as e:
            c()
        assert e.value.status == 4


def test_workspace_that_is_missing_or_too_small(pg):
    # nothing is enqueued: the output keeps what it held
    stream = torch.cuda.Stream()
    M, D, F, E, k = 5, 40, 24, 6, 2
    x, router, w, down = moe_case(3, "f16", M, D, F, E)
    y = torch.full((M, D), 7.0, dtype=torch.float16, device="cuda")
    need = pg.serve.moe_workspace_bytes(M, E, D, F, k)
    room = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    L, h = pg.lib(), ctypes.c_void_p(stream.cuda_stream)

    def moe():
        return L.pgemm_f16_moe(x.data_ptr(), router.data_ptr(), w.data_ptr(), down.data_ptr(), y.data_ptr(), None, None, M, E,
                               D, F, k, 1, 0, h)
    assert moe() == 9
    assert L.pgemm_set_workspace(h, room.data_ptr(), need - 1) == 0
    assert moe() == 9
    torch.cuda.synchronize()
    assert (y == 7).all()
    assert L.pgemm_set_workspace(h, room.data_ptr(), need) == 0
    room.fill_(0xFF)  # what it holds does not matter
    torch.cuda.synchronize()
    assert moe() == 0
    torch.cuda.synchronize()
    check("y", y, ref.moe(x, router, w, down, k, "silu", True)[0])
    assert L.pgemm_set_workspace(h, None, 0) == 0


@pytest.mark.parametrize("fmt", FMT)
def test_outputs_of_the_callers_own(pg, fmt):
    x, w, s = i8_case(4, fmt, 9, 40, 50, True)
    q, xs = call(pg, fmt, "quant_i8", x)
    oq, os_ = torch.full_like(q, 99), torch.full_like(xs, math.nan)
    got = call(pg, fmt, "quant_i8", x, q=oq, scale=os_)
    assert got[0] is oq and got[1] is os_ and torch.equal(oq, q) and torch.equal(os_, xs)

    def same(name, args, kw, shape, dtype=TYPES[fmt], key="out"):
        out = torch.full(shape, 77, dtype=dtype, device="cuda")
        assert call(pg, fmt, name, *args, **kw, **{key: out}) is out
        assert torch.equal(out, call(pg, fmt, name, *args, **kw))
    same("i8", (x, w, s), {}, (9, 80))
    same("i8", (q, w, s), dict(xs=xs), (9, 80))
    same("i8_gated", (x, w, s), dict(act="gelu"), (9, 40))
    m = moe_case(5, fmt, 9, 33, 20, 5)
    same("moe", (*m, 3), dict(act="gelu"), (9, 33))
    z, u = randn(torch.Generator().manual_seed(6), 9, 500).to(TYPES[fmt]).cuda(), torch.rand(9, device="cuda")
    same("sample", (z, u), {}, (9,), torch.int64, "token")


# ------------------------------------------------------------ empty

@pytest.mark.parametrize("fmt", FMT)
def test_empty(pg, fmt):
    t = TYPES[fmt]

    def z(*shape, dtype=t):
        return torch.zeros(shape, dtype=dtype, device="cuda")
    for M, K in ((0, 8), (5, 0), (0, 0)):
        q, s = call(pg, fmt, "quant_i8", z(M, K))
        assert q.shape == (M, ref.width(K)) and (s == 2.0 ** -126).all()
    for M, N, K in ((0, 5, 8), (5, 0, 8), (3, 6, 0), (300, 6, 0), (0, 0, 0)):
        w, s = z(2 * N, ref.width(K), dtype=torch.int8), torch.ones(2 * N, device="cuda")
        for name, cols in (("i8", 2 * N), ("i8_gated", N)):
            y = call(pg, fmt, name, z(M, K), w, s)
            assert y.shape == (M, cols) and not y.any()
            y = call(pg, fmt, name, z(M, ref.width(K), dtype=torch.int8), w, s, xs=torch.ones(M, device="cuda"))
            assert y.shape == (M, cols) and not y.any()
    for M, D, F in ((0, 8, 8), (5, 8, 0), (5, 0, 8), (70, 0, 0)):
        y, experts, weights = call(pg, fmt, "moe", z(M, D), z(4, D), z(4, 2 * F, D), z(4, D, F), 3, routing=True)
        assert y.shape == (M, D) and not y.any()
        # equal logits: the first experts, with the same weight each
        assert (experts == torch.arange(3, device="cuda")).all() and torch.equal(weights, torch.full_like(weights, 1 / 3))
    assert call(pg, fmt, "sample", z(0, 8), torch.zeros(0, device="cuda")).shape == (0,)
    assert (call(pg, fmt, "sample", z(3, 0), torch.zeros(3, device="cuda")) == -1).all()


# ------------------------------------------------------------ 8-bit integers

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("K", [5, 100, 1500, 9000])
def test_quant_ties_and_ranges(pg, fmt, K):
    # halves of a scale that is a power of two, either parity and sign; the type's largest and smallest values; zeros
    t = TYPES[fmt]
    rows = []
    halves = (torch.arange(K) % 253 - 126) / 2.0
    for scale in (1.0, 2.0 ** -8, 2.0 ** 8):
        r = halves * scale
        r[0] = 127 * scale
        rows.append(r)
    gen = torch.Generator().manual_seed(K)
    top, least = torch.finfo(t).max, torch.finfo(t).tiny * torch.finfo(t).eps
    rows += [torch.rand(K, generator=gen) * top, (torch.randint(-300, 301, (K,), generator=gen) * least), torch.zeros(K)]
    rows[3][0] = -top
    x = torch.stack(rows).to(t).cuda()
    q, s = call(pg, fmt, "quant_i8", x)
    want = ref.quant(x)
    assert torch.equal(s, want[1])
    equal("q", q, want[0])
    assert q.min() >= -127


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("K", [6, 50, 1200, 5000])
def test_quant_of_infinities_and_nan(pg, fmt, K):
    x = randn(torch.Generator().manual_seed(7), 5, K).to(TYPES[fmt]).cuda()
    for row, v in ((0, math.nan), (2, math.inf), (4, -math.inf)):
        x[row, K - 1] = v
    q, s = call(pg, fmt, "quant_i8", x)
    want = ref.quant(x)
    assert torch.equal(torch.isnan(s), torch.tensor([True, False, True, False, True], device="cuda"))
    equal("q", q, want[0])
    assert not q[::2].any() and torch.equal(s[1::2], want[1][1::2])
    # the row's products are NaN, the others' are not touched
    w, ws = torch.ones(20, ref.width(K), dtype=torch.int8, device="cuda"), torch.ones(20, device="cuda")
    for rows in ([0, 1], [0, 1, 2, 3, 4]):  # tokens that a workgroup makes integers of itself, and more
        y = call(pg, fmt, "i8", x[rows].contiguous(), w, ws)
        assert torch.isnan(y).all(1).tolist() == [r % 2 == 0 for r in rows] and torch.isfinite(y[1::2]).all()


@pytest.mark.parametrize("M,K", [(3000001, 5), (300001, 24), (40001, 1100), (17001, 4100)])
def test_quant_more_rows_than_a_launch_has_groups(pg, M, K):
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(K), device="cuda").half()
    q, s = pg.pgemm_f16_quant_i8(x)
    want = ref.quant(x)
    assert torch.equal(s, want[1])
    equal("q", q, want[0])


def test_quant_offsets_past_32_bits(pg):
    M, K = 70001, 65540
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(23)
    for m in range(0, M, 5000):
        x[m:m + 5000] = torch.randn(min(5000, M - m), K, generator=gen, device="cuda")
    q, s = pg.pgemm_bf16_quant_i8(x)
    some = [0, 1, 32767, 32768, 65535, 70000]
    want = ref.quant(x[some])
    assert torch.equal(s[some], want[1])
    equal("q", q[some], want[0])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [3, 20, 300])
def test_i8_largest_sums(pg, fmt, M):
    # -128 times -128 over the longest K: 2^31 - 2^18; scales whose product the type holds, though neither order of
    # multiplication keeps all partial products in fp32
    K = (1 << 17) - 16
    q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((4, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    q[1, ::2] = 127
    xs = torch.full((M,), 2.0 ** -40, device="cuda")
    xs[0], xs[1], xs[2] = 2.0 ** 100, 2.0 ** -126, 2.0 ** -149
    ws = torch.tensor([2.0 ** 9, 2.0 ** -130, 2.0 ** 95, 2.0 ** 118], device="cuda")
    want = ref.i8(q, xs, w, ws, TYPES[fmt])
    check_range("y", call(pg, fmt, "i8", q, w, ws, xs=xs), *want)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K", [(300, 128, 16384), (257, 127, 9000), (260, 1030, 3333), (513, 65, 100), (1000, 300, 4099),
                                   (2600, 2600, 33)])
def test_i8_tiles(pg, fmt, M, N, K):
    # pieces of K, ragged edges, large tiles with the rest in small ones
    x, w, ws = i8_case(M + N + K, fmt, M, N, K, False)
    q, xs = ref.quant(x)
    check("y", call(pg, fmt, "i8", x, w, ws), ref.i8(q, xs, w, ws, TYPES[fmt]))
    x, w, ws = i8_case(M + N + K, fmt, M, N, K, True)
    check("h", call(pg, fmt, "i8_gated", x, w, ws), ref.i8(q, xs, w, ws, TYPES[fmt], "silu"))


def test_i8_offsets_past_32_bits(pg):
    # weights of 4.4e9 bytes; the last rows are compared
    N, K = 66000, 66560
    gen = torch.Generator(device="cuda").manual_seed(8)
    w = torch.empty(N, K, dtype=torch.int8, device="cuda")
    for n in range(0, N, 6000):
        w[n:n + 6000] = torch.randint(-127, 128, (min(6000, N - n), K), generator=gen, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=gen, device="cuda") * 1e-4
    some = torch.cat([torch.arange(40), torch.arange(N - 40, N)]).cuda()
    for M in (2, 20, 300):
        q = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
        xs = torch.rand(M, generator=gen, device="cuda")
        y = pg.pgemm_bf16_i8(q, w, ws, xs=xs)
        check("y", y[:, some], ref.i8(q, xs, w[some], ws[some], torch.bfloat16))


# ------------------------------------------------------------ mixture of experts

@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,D", [(8, 40), (40, 40), (200, 72), (700, 24)])
def test_moe_ties(pg, fmt, E, D):
    # equal router rows have equal logits, to the last bit: the lowest index first
    x, router, w, down = moe_case(9, fmt, 7, D, 16, E)
    router[E // 2:] = router[:E - E // 2].clone()
    x[3] = 0
    k = min(E, 6)
    got = call(pg, fmt, "moe", x, router, w, down, k, routing=True)
    check_moe(got, ref.moe(x, router, w, down, k, "silu", True))
    assert got[1][3].tolist() == list(range(k))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [1, 30])
def test_moe_what_is_not_chosen(pg, fmt, M):
    # infinities and NaN in the experts that a token does not choose, or in other tokens, stay out of its result
    D, F, E, k = 72, 40, 12, 2
    x, router, w, down = moe_case(10, fmt, M, D, F, E)
    clean = call(pg, fmt, "moe", x, router, w, down, k, routing=True)
    for e, v in ((0, math.nan), (5, math.inf), (7, -math.inf)):
        w[e, 3], down[e, 5] = v, v
    touched = torch.isin(clean[1], torch.tensor([0, 5, 7], device="cuda")).any(1)
    y, experts, weights = call(pg, fmt, "moe", x, router, w, down, k, routing=True)
    assert torch.equal(experts, clean[1]) and torch.equal(weights, clean[2])
    assert torch.equal(y[~touched], clean[0][~touched]) and not torch.isfinite(y[touched]).all()
    if M > 1:
        x, router, w, down = moe_case(10, fmt, M, D, F, E)
        x[4, 7], x[9, 0] = math.nan, math.inf
        y, experts, weights = call(pg, fmt, "moe", x, router, w, down, k, routing=True)
        others = torch.tensor([m for m in range(M) if m not in (4, 9)], device="cuda")
        assert torch.equal(y[others], clean[0][others]) and torch.isnan(y[4]).all() and torch.isnan(weights[4]).all()
        assert ((experts >= 0) & (experts < E)).all()


@pytest.mark.parametrize("fmt", FMT)
def test_moe_router_with_nan_and_infinities(pg, fmt):
    # a logit that is NaN comes last; with an infinite one the weights are NaN, as a softmax's
    D, F, E = 16, 8, 5
    x, router, w, down = moe_case(11, fmt, 4, D, F, E)
    x.abs_()
    router[1] = math.nan
    _, experts, weights = call(pg, fmt, "moe", x, router, w, down, 4, routing=True)
    assert not (experts == 1).any() and torch.isfinite(weights).all()
    _, experts, weights = call(pg, fmt, "moe", x, router, w, down, 5, routing=True)
    assert (experts[:, 4] == 1).all() and torch.isnan(weights).all()
    router[1], router[3] = 0, math.inf
    _, experts, weights = call(pg, fmt, "moe", x, router, w, down, 2, routing=True)
    assert (experts[:, 0] == 3).all() and torch.isnan(weights).all()


@pytest.mark.parametrize("M,F", [(1, 64), (9, 5), (9, 200), (60, 333)])
def test_moe_hidden_values_past_f16(pg, M, F):
    # hidden values to 1e9 and of 1e-9 in the same layer, results inside f16
    D, E, k = 48, 4, 2
    x, router, w, down = moe_case(12, "f16", M, D, F, E)
    w[0] *= 4000.0
    down[0] *= 2.0 ** -14
    w[1] *= 2.0 ** -12
    down[1] *= 1000.0
    got = pg.pgemm_f16_moe(x, router, w, down, k, routing=True)
    want = ref.moe(x, router, w, down, k, "silu", True)
    equal("experts", got[1], want[1])
    check_range("y", got[0], *want[0])
    assert torch.isfinite(got[0]).all()


@pytest.mark.parametrize("fmt", FMT)
def test_moe_all_tokens_to_one_expert(pg, fmt):
    # more tokens of an expert than a workgroup takes at a time, and experts with none
    for M, E in ((64, 40), (50, 3), (150, 64), (17, 30)):
        x, router, w, down = moe_case(13, fmt, M, 40, 24, E)
        x.abs_()
        router[2] = 1.0
        got = call(pg, fmt, "moe", x, router, w, down, 1, normalize=False, routing=True)
        assert (got[1] == 2).all()
        check_moe(got, ref.moe(x, router, w, down, 1, "silu", False))


def test_moe_offsets_past_32_bits(pg):
    # 2.3e9 values in each of the experts' matrices
    M, D, F, E, k = 3, 4096, 4480, 64, 64 // 8
    gen = torch.Generator(device="cuda").manual_seed(14)
    x = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
    router = (torch.randn(E, D, generator=gen, device="cuda") * D ** -0.5).bfloat16()
    w = torch.empty(E, 2 * F, D, dtype=torch.bfloat16, device="cuda")
    down = torch.empty(E, D, F, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = torch.randn(2 * F, D, generator=gen, device="cuda") * D ** -0.5
        down[e] = torch.randn(D, F, generator=gen, device="cuda") * F ** -0.5
    router[E - 1] = x.float().mean(0).bfloat16()  # the last expert is chosen too
    got = pg.pgemm_bf16_moe(x, router, w, down, k, routing=True)
    assert (got[1] == E - 1).any()
    check_moe(got, ref.moe(x, router, w, down, k, "silu", True))


# ------------------------------------------------------------ sampling

def sampled(pg, fmt, z, u, **kw):
    return call(pg, fmt, "sample", z.to(TYPES[fmt]).cuda(), u.cuda(), **{k: None if v is None else v.cuda() for k, v in kw.items()}).cpu()


@pytest.mark.parametrize("fmt", FMT)
def test_sample_masks(pg, fmt):
    V = 3000
    z = randn(torch.Generator().manual_seed(15), 6, V, scale=2.0)
    z[0] = -math.inf                       # nothing left
    z[1] = -math.inf
    z[1, 2999] = torch.finfo(TYPES[fmt]).min  # one token, the type's lowest value
    z[2, 1:] = -math.inf
    z[3, 100] = math.nan
    z[4, 7], z[4, 2000] = math.inf, math.inf  # they share all of the probability
    z[5] = torch.finfo(TYPES[fmt]).min
    for u in (0.0, 0.3, 0.999999):
        u = torch.full((6,), u)
        got = sampled(pg, fmt, z, u)
        assert got.tolist()[:5] == [-1, 2999, 0, -1, 7 if u[0] < 0.5 else 2000]
        assert got[5] == int(u[5].double() * V)
        equal("token", got, ref.sample(z.to(TYPES[fmt]), u))
        for t in (1e-30, 0.01, 1e30, math.inf):
            t = torch.full((6,), t)
            equal("token", sampled(pg, fmt, z, u, temperature=t), ref.sample(z.to(TYPES[fmt]), u, temperature=t))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("V", [1, 63, 5000, 65535, 65536, 200001])
def test_sample_equal_logits(pg, fmt, V):
    # uniform: the u V-th token; more than 16 bits' worth of one value are counted otherwise
    M = 9
    u = torch.rand(M, generator=torch.Generator().manual_seed(V))
    for value in (0.0, -0.0, 3.0, -7.0):
        z = torch.full((M, V), value)
        got = sampled(pg, fmt, z, u)
        assert got.tolist() == [int(x) for x in (u.double() * V).floor()]
    # either zero, in the order of the indices; the token below comes last
    z = torch.zeros(M, V)
    z[:, ::2] = -0.0
    assert sampled(pg, fmt, z, u).tolist() == [int(x) for x in (u.double() * V).floor()]
    k = torch.full((M,), 3, dtype=torch.int32)
    assert sampled(pg, fmt, z, u, top_k=k).tolist() == [int(x) for x in (u.double() * min(V, 3)).floor()]


@pytest.mark.parametrize("fmt", FMT)
def test_sample_counts_past_16_bits(pg, fmt):
    # most of a row at one value, others above and below it; all settings
    gen = torch.Generator().manual_seed(16)
    V, M = 210000, 12
    z = torch.full((M, V), -1.0)
    at = torch.randperm(V, generator=gen)[:30000]
    z[:, at] = randn(gen, M, 30000, scale=3.0)
    u = torch.rand(M, generator=gen)
    t, k, p, q = settings(gen, M)
    k[::3] *= 2000
    for kw in ({}, dict(temperature=t, top_k=k, top_p=p, min_p=q), dict(top_p=p), dict(temperature=t.clamp(min=0.5), min_p=q)):
        equal("token", sampled(pg, fmt, z, u, **kw), ref.sample(z.to(TYPES[fmt]), u, **kw))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("V", [300, 65601, 140001])
def test_sample_masked_by_the_lowest_value(pg, fmt, V):
    gen = torch.Generator().manual_seed(V)
    M = 12
    low = torch.finfo(TYPES[fmt]).min
    z = torch.full((M, V), low)
    for m in range(1, M):  # row 0 has nothing else
        at = torch.randperm(V, generator=gen)[:2 ** m // 4 + 1]
        z[m, at] = randn(gen, len(at), scale=low / -9 if m % 3 else 2.0)  # to half of the type's range, or ordinary logits
    z[5, torch.randperm(V, generator=gen)[:V // 3]] = -math.inf
    u = torch.rand(M, generator=gen)
    u[3:6] = 1 - 2.0 ** -24
    t, k, p, q = settings(gen, M)
    k[::2] = V // 2 + 7
    for T in (1.0, 0.01, -low / 30, -low * 100 if fmt == "f16" else math.inf, math.inf):
        T = torch.full((M,), T)
        for kw in ({}, dict(top_k=k), dict(top_p=p), dict(min_p=q), dict(top_k=k, top_p=p, min_p=q)):
            equal(f"T {T[0]} {list(kw)}", sampled(pg, fmt, z, u, temperature=T, **kw), ref.sample(z.to(TYPES[fmt]), u, temperature=T, **kw))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("V", [40, 3001])
def test_sample_limits_of_settings(pg, fmt, V):
    gen = torch.Generator().manual_seed(17)
    M = 16
    z = randn(gen, M, V, scale=2.0)
    t = TYPES[fmt]
    u = torch.rand(M, generator=gen)
    u[:3] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5])

    def full(v, dtype=torch.float32):
        return torch.full((M,), v, dtype=dtype)
    first = ref.sample(z.to(t), u, temperature=torch.zeros(M))
    for kw in (dict(temperature=full(0.0)), dict(temperature=full(1e-45)), dict(top_k=full(1, torch.int32)), dict(top_p=full(0.0)),
               dict(top_p=full(-3.0)), dict(top_p=full(1e-30)), dict(min_p=full(2.0)), dict(min_p=full(math.inf))):
        equal(str(kw), sampled(pg, fmt, z, u, **kw), first)
    free = ref.sample(z.to(t), u)
    for kw in ({}, dict(temperature=full(1.0)), dict(top_k=full(0, torch.int32)), dict(top_k=full(-5, torch.int32)),
               dict(top_k=full(2 ** 31 - 1, torch.int32)), dict(top_p=full(1.0)), dict(top_p=full(math.inf)), dict(min_p=full(0.0)),
               dict(min_p=full(-1.0))):
        equal(str(kw), sampled(pg, fmt, z, u, **kw), free)
    # an infinite temperature makes all tokens alike, in their order
    equal("hot", sampled(pg, fmt, z, u, temperature=full(math.inf)), ref.sample(z.to(t), u, temperature=full(math.inf)))
    # outside [0, 1): the nearest
    last = ref.sample(z.to(t), full(1.0), top_k=full(7, torch.int32))
    equal("above", sampled(pg, fmt, z, full(5.0), top_k=full(7, torch.int32)), last)
    equal("below", sampled(pg, fmt, z, full(-1.0)), first)
    for kw in (dict(temperature=full(-1.0)), dict(temperature=full(math.nan)), dict(top_p=full(math.nan)), dict(min_p=full(math.nan))):
        assert (sampled(pg, fmt, z, u, **kw) == -1).all(), kw
    assert (sampled(pg, fmt, z, full(math.nan)) == -1).all()


@pytest.mark.parametrize("fmt", FMT)
def test_sample_all_values_of_the_type(pg, fmt):
    # every value there is but NaN, once and in any order: as many as there are counters
    t = TYPES[fmt]
    v = torch.arange(-32768, 32768).to(torch.int16).view(t)
    v = v[~torch.isnan(v)]
    v = v[(v < 1e4) & (v > -1e4)]
    gen = torch.Generator().manual_seed(18)
    M = 8
    z = torch.stack([v[torch.randperm(len(v), generator=gen)] for _ in range(M)])
    u = torch.rand(M, generator=gen)
    for T in (0.7, 50.0, 5000.0, 1e6):
        temperature = torch.full((M,), T)
        equal(f"T {T}", sampled(pg, fmt, z, u, temperature=temperature), ref.sample(z, u, temperature=temperature))
        for kw in (dict(top_k=torch.full((M,), 30000, dtype=torch.int32)), dict(top_p=torch.full((M,), 0.9)), dict(min_p=torch.full((M,), 0.3))):
            equal(f"T {T} {kw}", sampled(pg, fmt, z, u, temperature=temperature, **kw), ref.sample(z, u, temperature=temperature, **kw))


@pytest.mark.parametrize("fmt", FMT)
def test_sample_shared_settings(pg, fmt):
    gen = torch.Generator().manual_seed(19)
    M, V = 30, 900
    z, u = randn(gen, M, V, scale=2.0), torch.rand(M, generator=gen)
    one = dict(temperature=torch.tensor(0.7), top_k=torch.tensor(40, dtype=torch.int32), top_p=torch.tensor(0.9), min_p=torch.tensor(0.01))
    want = ref.sample(z.to(TYPES[fmt]), u, **one)
    equal("all shared", sampled(pg, fmt, z, u, **one), want)
    for key in one:
        equal(key, sampled(pg, fmt, z, u, **{**one, key: one[key].expand(M).contiguous()}), want)


def test_sample_frequencies(pg):
    # evenly spread u visit each token as often as its probability says, to one visit
    V, M = 50, 20000
    z = randn(torch.Generator().manual_seed(20), 1, V, scale=1.5).bfloat16()
    u = (torch.arange(M) + 0.5) / M
    got = pg.pgemm_bf16_sample(z.expand(M, V).contiguous().cuda(), u.cuda()).cpu()
    p = torch.softmax(z[0].double(), 0)
    assert ((torch.bincount(got, minlength=V) - p * M).abs() <= 1 + 1e-3).all()


def test_sample_offsets_past_32_bits(pg):
    M, V = 17000, 131077
    gen = torch.Generator(device="cuda").manual_seed(21)
    z = torch.empty(M, V, dtype=torch.bfloat16, device="cuda")
    for m in range(0, M, 2000):
        z[m:m + 2000] = torch.randn(min(2000, M - m), V, generator=gen, device="cuda") * 2
    u = torch.rand(M, generator=gen, device="cuda")
    k = torch.tensor(30, dtype=torch.int32, device="cuda")
    got = pg.pgemm_bf16_sample(z, u, top_k=k)
    some = [0, 1, 16383, 16384, 16999]
    equal("token", got[some].cpu(), ref.sample(z[some].cpu(), u[some].cpu(), top_k=k.cpu()))


@pytest.mark.parametrize("fmt", FMT)
def test_sample_more_rows_than_workgroups(pg, fmt):
    # a workgroup's second row, after one of any kind (taken, refused, greedy): the same tokens as the first time
    gen = torch.Generator().manual_seed(24)
    n, V = 65536, 70
    z, u = randn(gen, n, V, scale=2.0), torch.rand(n, generator=gen)
    t = torch.rand(n, generator=gen) * 2
    z[::7] = -math.inf
    z[3::11, 5] = math.nan
    t[::5] = 0
    turn = torch.randperm(n, generator=gen)
    got = sampled(pg, fmt, torch.cat([z, z[turn]]), torch.cat([u, u[turn]]), temperature=torch.cat([t, t[turn]]))
    assert torch.equal(got[n:], got[:n][turn])
    some = torch.cat([torch.arange(200), torch.arange(n - 200, n)])
    equal("token", got[some], ref.sample(z[some].to(TYPES[fmt]), u[some], temperature=t[some]))


# ------------------------------------------------------------ together

def serving_step(pg, fmt, x, experts, head, u, some):
    """Tokens through an expert layer, a vocabulary head in 8 bits and the choice of the next token."""
    y, chosen, p = call(pg, fmt, "moe", x, *experts, 2, routing=True)
    h = call(pg, fmt, "i8_gated", y, *head[0], act="gelu")
    q, s = call(pg, fmt, "quant_i8", h)
    z = call(pg, fmt, "i8", q, *head[1], xs=s)
    return y, chosen, p, h, z, call(pg, fmt, "sample", z, u, *some)


def serving_case(pg, fmt, seed, M, D=72, F=40, E=6, V=1000):
    gen = torch.Generator().manual_seed(seed)
    x, *experts = moe_case(seed, fmt, M, D, F, E)
    def packed(n, k):
        return call(pg, fmt, "quant_i8", randn(gen, n, k, scale=2 * k ** -0.5).to(TYPES[fmt]).cuda())
    return x, experts, (packed(2 * 48, D), packed(V, 48)), torch.rand(M, generator=gen).cuda(), on_gpu(*settings(gen, M))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [1, 7, 100, 300])
def test_a_serving_step(pg, fmt, M):
    x, experts, head, u, some = serving_case(pg, fmt, 22 + M, M)
    y, chosen, p, h, z, token = serving_step(pg, fmt, x, experts, head, u, some)
    check_moe((y, chosen, p), ref.moe(x, *experts, 2, "silu", True))
    q, xs = ref.quant(y)
    check("h", h, ref.i8(q, xs, *head[0], TYPES[fmt], "gelu"))
    q, xs = ref.quant(h)
    check("z", z, ref.i8(q, xs, *head[1], TYPES[fmt]))
    equal("token", token.cpu(), ref.sample(z.cpu(), u.cpu(), *[t.cpu() for t in some]))
    for a, b in zip(serving_step(pg, fmt, x, experts, head, u, some), (y, chosen, p, h, z, token)):
        assert torch.equal(a, b)  # the same bits every time


@pytest.mark.parametrize("fmt", FMT)
def test_other_streams(pg, fmt):
    case = serving_case(pg, fmt, 30, 90)
    here = serving_step(pg, fmt, *case)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):  # side by side, each with a workspace of its own
        for s in streams:
            with torch.cuda.stream(s):
                got.append(serving_step(pg, fmt, *case))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, here):
            assert torch.equal(a, b)
    x, experts = case[:2]
    y = call(pg, fmt, "moe", x, *experts, 2, stream=streams[0])
    z = call(pg, fmt, "i8", x, *call(pg, fmt, "quant_i8", experts[0], stream=streams[0]), stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, here[0]) and z.shape == (90, 6)
    for s in streams:
        pg.release_workspace(s)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [3, 70])
def test_graph(pg, fmt, M):
    # two graphs of a step, replayed in turn on other inputs, with eager calls of larger ones in between
    x, experts, head, u, some = serving_case(pg, fmt, 31, M)

    def step():
        return serving_step(pg, fmt, x, experts, head, u, some)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for turn in range(4):
        gen = torch.Generator().manual_seed(40 + turn)
        x.copy_(randn(gen, *x.shape).to(x.dtype))
        u.copy_(torch.rand(M, generator=gen))
        want = [t.clone() for t in step()]
        big = serving_case(pg, fmt, 50 + turn, 200 + 100 * turn, D=104, F=72)
        serving_step(pg, fmt, *big)
        junk = [torch.full((1 << 20,), math.nan, device="cuda") for _ in range(4)]
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)
        del junk
    pg.release_workspace(side)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_example_serves(pg, bits, temperature):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import gated_lm
    gen = torch.Generator().manual_seed(60)
    embed, block, head = (randn(gen, n, k, scale=k ** -0.5).cuda() for n, k in ((300, 64), (192, 64), (300, 96)))
    first = torch.arange(7, device="cuda")
    got = gated_lm.serve(embed, block, head, first, 5, bits, temperature)
    assert got.shape == (7, 5) and got.dtype == torch.int64 and ((got >= 0) & (got < 300)).all()
    assert torch.equal(got, gated_lm.serve(embed, block, head, first, 5, bits, temperature))
