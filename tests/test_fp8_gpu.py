"""8-bit floating point products with a scale for each block of 128 and the
quantization of their operands, against their definitions.

Codes and scales are functions of the inputs alone and have to be equal. A
product's tolerance counts roundings, each at most half a step (2^-24 in fp32) but
those inside the tensor cores, which may truncate (2^-23): at most 128 additions in
a block, K/128 products by a factor (itself two roundings) and as many additions,
the joining of as many parts; all relative to the sum of magnitudes, A:
(2 128 + 4 K/128 + 4) 2^-24 A. A bf16 output adds 2^-8 of itself.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

import memory_bound_weight_gb300 as mbw  # noqa: E402

E4M3 = torch.float8_e4m3fn
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def divided(most):  # by a tensor: torch multiplies by the reciprocal of a number
    return most / torch.full_like(most, 448.0)


def plain_rows(x):
    """The definition, in elementary steps: codes and scales of rows."""
    m, k = x.shape
    y = x.float().view(m, k // 128, 128)
    s = divided(y.abs().amax(-1))
    q = torch.where(s[..., None] == 0, torch.zeros_like(y), y / s[..., None])
    return q.to(E4M3).view(m, k), s


def plain_blocks(w):
    n, k = w.shape
    y = torch.nn.functional.pad(w.float(), (0, 0, 0, -n % 128)).view(-1, 128, k // 128, 128)
    s = divided(y.abs().amax((1, 3)))
    q = torch.where(s[:, None, :, None] == 0, torch.zeros_like(y), y / s[:, None, :, None])
    return q.to(E4M3).view(-1, k)[:n], s


def same(a, b):
    """Equal, a NaN to a NaN of either sign."""
    x, y = a.float(), b.float()
    return bool(((x == y) | (x.isnan() & y.isnan())).all())


def operands(g, m, n, k):
    x = torch.randn(m, k, generator=g, device="cuda") * torch.exp(torch.randn(k, generator=g, device="cuda"))
    w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5 * torch.exp(torch.randn(n, 1, generator=g, device="cuda"))
    return (*plain_rows(x.bfloat16()), *plain_blocks(w.bfloat16()))


def exact(x, xs, w, ws):
    """The product in 64 bits, and the sum of magnitudes."""
    k, n = x.shape[1], w.shape[0]
    xd = x.double() * xs.double().repeat_interleave(128, 1)
    wd = w.double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:n]
    return xd @ wd.T, xd.abs() @ wd.abs().T, (2 * 128 + 4 * k / 128 + 4) * 2.0 ** -24


def half_step(y):
    return y.abs() * 2.0 ** -8 + 2.0 ** -133


def check(got, want, tol, what=""):
    err = (got.double() - want).abs()
    ok = err <= tol * (1 + 2.0 ** -7)  # the output's rounding is relative to the rounded sum
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()}, worst {float((err / tol.clamp_min(1e-300)).max())}"


SIZES = [(1, 1, 128), (1, 2048, 2048), (2, 7, 256), (3, 128, 128), (5, 129, 640), (15, 300, 1152), (16, 1000, 3584), (17, 100, 384),
         (31, 257, 5120), (33, 2560, 896), (64, 64, 4096), (65, 513, 1280), (100, 18944, 256), (128, 128, 18944), (129, 130, 128),
         (130, 1, 512), (200, 1031, 768), (256, 256, 256), (257, 4608, 3584), (500, 127, 2560), (777, 640, 1408), (1025, 385, 128)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k):
    x, xs, w, sc = operands(gen(m * 7 + n + k), m, n, k)
    y, mass, eps = exact(x, xs, w, sc)
    got = mbw.gemm_fp8_b128(x, xs, w, sc)
    check(got, y, mass * eps + half_step(y), "bf16")
    assert torch.equal(mbw.gemm_fp8_b128(x, xs, w, sc, workspace=torch.empty(64, device="cuda")), got)  # the same again
    with mbw.output_fp32():
        check(mbw.gemm_fp8_b128(x, xs, w, sc), y, mass * eps + 2.0 ** -149, "fp32")


@pytest.mark.parametrize("m,n,k", SIZES[::2] + [(40, 5632, 2048)])
def test_gated_product_with_a_residual(m, n, k):
    g = gen(m + 3 * n + k)
    x, xs, w, sc = operands(g, m, n, k)
    _, _, u, su = operands(g, 1, n, k)
    r = torch.randn(m, n, generator=g, device="cuda").bfloat16()
    a, mass_a, eps = exact(x, xs, w, sc)
    b, mass_b, _ = exact(x, xs, u, su)
    act = a * torch.sigmoid(a)
    # |silu'| <= 1.1; silu in fp32: exp within 2 steps (2^-22) of an argument that is itself rounded, which acts as a
    # change of a by 2^-24, a sum, a quotient: 2^-21; the product and the sum with the residual 2^-24 each
    tol = 1.1 * mass_a * eps * b.abs() + act.abs() * mass_b * eps + 1.1 * mass_a * mass_b * eps * eps
    tol = tol + (act * b).abs() * 2.0 ** -20 + r.double().abs() * 2.0 ** -23
    want = act * b + r.double()
    got = mbw.gemm_fp8_b128(x, xs, w, sc, residual=r, up_weights=u, up_scales=su)
    check(got, want, tol + half_step(want), "gated, residual")
    check(mbw.gemm_fp8_b128(x, xs, w, sc, up_weights=u, up_scales=su), act * b, tol + half_step(act * b), "gated")
    # the residual may be the output
    y, mass, eps = exact(x, xs, w, sc)
    out = r.clone()
    assert mbw.gemm_fp8_b128(x, xs, w, sc, out=out, residual=out) is out
    want = y + r.double()
    check(out, want, mass * eps + want.abs() * 2.0 ** -24 + half_step(want), "in place")


FEW = [(9, 9001, 2560), (16, 2560, 9728), (17, 3584, 1024), (24, 20011, 640), (32, 1000, 9728), (33, 2050, 1280), (61, 5632, 2048), (64, 21000, 384), (64, 1000, 9728),
       (65, 20480, 512), (90, 300, 18944), (127, 2049, 1792), (128, 19600, 640), (128, 3584, 3584)]


@pytest.mark.parametrize("m,n,k", FEW)
def test_few_rows_of_larger_matrices(m, n, k):
    """Weights of more than one tile a CTA, of one, and cut along k; residuals on any bytes that a tensor of bf16 lies on."""
    g = gen(m + n + 5 * k)
    x, xs, w, sc = operands(g, m, n, k)
    _, _, u, su = operands(g, 1, n, k)
    y, mass, eps = exact(x, xs, w, sc)
    z, mass_z, _ = exact(x, xs, u, su)
    check(mbw.gemm_fp8_b128(x, xs, w, sc), y, mass * eps + half_step(y), "bf16")
    with mbw.output_fp32():
        check(mbw.gemm_fp8_b128(x, xs, w, sc), y, mass * eps + 2.0 ** -149, "fp32")
    act = y * torch.sigmoid(y)  # the tolerance is derived in test_gated_product_with_a_residual
    tol = 1.1 * mass * eps * z.abs() + act.abs() * mass_z * eps + 1.1 * mass * mass_z * eps * eps + (act * z).abs() * 2.0 ** -20
    for off in (0, 1, 4):
        r = torch.randn(m * n + off, generator=g, device="cuda").bfloat16()[off:].view(m, n)
        want = y + r.double()
        check(mbw.gemm_fp8_b128(x, xs, w, sc, residual=r), want, mass * eps + want.abs() * 2.0 ** -24 + half_step(want), "residual")
        want = act * z + r.double()
        got = mbw.gemm_fp8_b128(x, xs, w, sc, residual=r, up_weights=u, up_scales=su)
        check(got, want, tol + r.double().abs() * 2.0 ** -23 + half_step(want), "gated, residual")
        assert torch.equal(got, mbw.gemm_fp8_b128(x, xs, w, sc, residual=r, up_weights=u, up_scales=su))
    out = r.clone()
    mbw.gemm_fp8_b128(x, xs, w, sc, out=out, residual=out)  # in place
    want = y + r.double()
    check(out, want, mass * eps + want.abs() * 2.0 ** -24 + half_step(want), "in place")


@pytest.mark.parametrize("m", [16, 33, 64, 100])
def test_gated_products_one_behind_the_other(m):
    """Every SM with a tile of its own, launches that overlap, a ring whose stages the issuing warps take in turn: always the same."""
    g = gen(m)
    n, k = 18944, 3584
    x, xs, w, sc = operands(g, m, n, k)
    _, _, u, su = operands(g, 1, n, k)
    first = mbw.gemm_fp8_b128(x, xs, w, sc, up_weights=u, up_scales=su)
    rest = [mbw.gemm_fp8_b128(x, xs, w, sc, up_weights=u, up_scales=su) for _ in range(40)]
    assert all(torch.equal(first, y) for y in rest)
    a, mass_a, eps = exact(x, xs, w[-384:], sc[-3:])
    b, mass_b, _ = exact(x, xs, u[-384:], su[-3:])
    want = a * torch.sigmoid(a) * b  # the tolerance is derived in test_gated_product_with_a_residual
    tol = 1.1 * mass_a * eps * b.abs() + (a * torch.sigmoid(a)).abs() * mass_b * eps + 1.1 * mass_a * mass_b * eps * eps
    check(first[:, -384:], want, tol + want.abs() * 2.0 ** -20 + half_step(want))


def test_no_rows_or_no_outputs():
    x, xs, w, sc = operands(gen(1), 4, 130, 256)
    assert mbw.gemm_fp8_b128(x[:0], xs[:0], w, sc).shape == (0, 130)
    assert mbw.gemm_fp8_b128(x, xs, w[:0], sc[:0]).shape == (4, 0)
    assert mbw.quantize_fp8_g128(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))[0].shape == (0, 256)
    assert mbw.quantize_fp8_b128(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))[1].shape == (0, 2)
    assert mbw.dequant_fp8_g128(x[:0], xs[:0]).shape == (0, 256)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_codes_of_every_kind_and_scales_far_apart(m):
    """All finite codes, among them the subnormal ones, with scales over many powers of two whose products cancel."""
    g = gen(m)
    n, k = 260, 640
    bits = torch.randint(0, 256, (m + n, k), generator=g, device="cuda").to(torch.uint8)
    bits[(bits & 0x7F) == 0x7F] = 0x81  # no NaN
    x, w = bits[:m].view(E4M3).clone(), bits[m:].view(E4M3).clone()
    xs = torch.exp2(torch.randint(-40, 40, (m, k // 128), generator=g, device="cuda").float()) * 1.1
    sc = torch.exp2(torch.randint(-40, 40, (3, k // 128), generator=g, device="cuda").float()) * 1.3
    y, mass, eps = exact(x, xs, w, sc)
    check(mbw.gemm_fp8_b128(x, xs, w, sc), y, mass * eps + half_step(y))
    # within a block: large terms that cancel, and a small one that remains
    x = torch.zeros(m, 128, device="cuda")
    x[:, 0], x[:, 77], x[:, 100] = 448.0, 448.0, 2.0 ** -9
    w = torch.zeros(n, 128, device="cuda")
    w[:, 0], w[:, 77], w[:, 100] = 448.0, -448.0, 1.0
    one = torch.ones(m, 1, device="cuda"), torch.ones(3, 1, device="cuda")
    y, mass, eps = exact(x.to(E4M3), one[0], w.to(E4M3), one[1])
    check(mbw.gemm_fp8_b128(x.to(E4M3), one[0], w.to(E4M3), one[1]), y, mass * eps + half_step(y), "cancelling")


@pytest.mark.parametrize("m,n", [(3, 300), (100, 300), (300, 500)])
def test_what_is_no_number_stays_in_its_row_and_column(m, n):
    k = 512
    x, xs, w, sc = operands(gen(m), m, n, k)
    y, mass, eps = exact(x, xs, w, sc)
    bits = x.view(torch.uint8).clone()
    bits[1, 200] = 0x7F
    xs2 = xs.clone()
    xs2[0, 3] = float("inf")
    wbits = w.view(torch.uint8).clone()
    wbits[n - 1, 5] = 0xFF
    got = mbw.gemm_fp8_b128(bits.view(E4M3), xs2, wbits.view(E4M3), sc)
    assert got[1].isnan().all() and got[:, n - 1].isnan().all()
    assert not got[0, :n - 1].isfinite().any()
    check(got[2:, :n - 1], y[2:, :n - 1], (mass * eps + half_step(y))[2:, :n - 1])


def test_rows_do_not_depend_on_the_rows_beside_them():
    """Without parts, a row's sums are taken in one order whatever the batch of its orientation."""
    x, xs, w, sc = operands(gen(5), 400, 700, 1024)
    for a, b in ((16, 3), (400, 130)):
        whole = mbw.gemm_fp8_b128(x[:a].contiguous(), xs[:a].contiguous(), w, sc)
        part = mbw.gemm_fp8_b128(x[:b].contiguous(), xs[:b].contiguous(), w, sc)
        assert torch.equal(whole[:b], part)


def test_rows_behind_the_last_are_left_as_they_were():
    """The output is part of a larger buffer; so are the operands, which end where the buffer does."""
    for m, n in ((3, 200), (70, 333), (200, 385)):
        x, xs, w, sc = operands(gen(m), m, n, 384)
        big = torch.full((m * n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[:m * n].view(m, n)
        mbw.gemm_fp8_b128(x, xs, w, sc, out=out)
        assert big[m * n:].eq(7).all()
        y, mass, eps = exact(x, xs, w, sc)
        check(out, y, mass * eps + half_step(y))


def test_captured_and_on_two_streams():
    sizes = [(1, 2048, 2048), (50, 700, 1152), (300, 1000, 512)]
    data = [operands(gen(i), *s) for i, s in enumerate(sizes)]
    want = [[mbw.gemm_fp8_b128(*d) for d in data] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = [mbw.gemm_fp8_b128(*d) for d in data]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    g = torch.cuda.CUDAGraph()
    h = torch.randn(50, 1152, device="cuda").bfloat16()
    with torch.cuda.graph(g):
        outs = [mbw.gemm_fp8_b128(*d) for d in data]
        q, qs = mbw.quantize_fp8_g128(h)
        chain = mbw.gemm_fp8_b128(q, qs, data[1][2], data[1][3])
    for _ in range(3):
        h.copy_(torch.randn(50, 1152, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[0]))
        x, xs = plain_rows(h)
        assert torch.equal(chain, mbw.gemm_fp8_b128(x, xs, data[1][2], data[1][3]))


# ------------------------------------------------------------ quantization ----
@pytest.mark.parametrize("m,k", [(1, 128), (1, 3584), (2, 256), (3, 384), (7, 18944), (61, 2560), (130, 128), (1000, 640), (5, 128 * 90)])
def test_quantizing_rows(m, k):
    g = gen(m + k)
    wide = (torch.randn(m, k + 24, generator=g, device="cuda") * torch.exp(2 * torch.randn(k + 24, generator=g, device="cuda"))).bfloat16()
    x = wide[:, 8:8 + k]  # rows of a wider matrix
    q, s = mbw.quantize_fp8_g128(x)
    want, scale = plain_rows(x)
    assert torch.equal(s, scale) and same(q, want)
    assert torch.equal(mbw.dequant_fp8_g128(q, s), q.float() * s.repeat_interleave(128, 1))
    wn = (1 + 0.3 * torch.randn(k, generator=g, device="cuda")).bfloat16()
    for eps in (1e-6, 0.0, 0.25):
        r = (1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + eps)).float()
        want, scale = plain_rows((x.float() * r * wn.float()).bfloat16())
        q, s = mbw.quantize_fp8_g128(x, norm_weight=wn, norm_eps=eps)
        assert torch.equal(s, scale) and same(q, want)


@pytest.mark.parametrize("n,k", [(1, 128), (127, 256), (128, 128), (129, 384), (1000, 1152), (300, 18944)])
def test_quantizing_weights(n, k):
    w = (torch.randn(n, k, generator=gen(n), device="cuda") * torch.exp(torch.randn(n, 1, generator=gen(k), device="cuda"))).bfloat16()
    q, s = mbw.quantize_fp8_b128(w)
    want, scale = plain_blocks(w)
    assert torch.equal(s, scale) and same(q, want)
    full = s.repeat_interleave(128, 1).repeat_interleave(128, 0)[:n]
    assert torch.equal(mbw.dequant_fp8_b128(q, s), q.float() * full)


def awkward():
    """Blocks of zeros, of the type's smallest and largest values, of one value, with a NaN or an infinity; every exponent."""
    x = torch.zeros(16, 384, device="cuda")
    x[1] = 1.0
    x[2] = 9.2e-41  # the smallest bf16
    x[3] = 3.38e38
    x[4, ::2] = 9.2e-41
    x[5] = torch.exp2(torch.linspace(-126, 126, 384, device="cuda"))
    x[6] = torch.exp2(torch.linspace(-30, 8, 384, device="cuda")) * 1.37
    x[7, 5] = float("nan")
    x[8, 130] = float("inf")
    x[9, 300] = -float("inf")
    x[10, :128] = torch.arange(128, device="cuda") * 2.0 ** -120
    x[11] = torch.linspace(-448, 448, 384, device="cuda")
    x[12] = torch.linspace(-1e-20, 1e-20, 384, device="cuda")
    x[13, 7], x[13, 8] = 1e-38, 3e38
    x[14] = -1.17e-38
    x[15] = torch.linspace(1e30, 2e30, 384, device="cuda")
    return x.bfloat16()


def test_quantizing_awkward_blocks():
    x = awkward()
    q, s = mbw.quantize_fp8_g128(x)
    want, scale = plain_rows(x)
    assert same(s, scale) and same(q, want)
    for row, block in ((7, 0), (8, 1), (9, 2)):
        v = mbw.dequant_fp8_g128(q, s)[row].view(3, 128)
        assert v[block].isnan().all() and v.isnan().sum() == 128
    for row in x:  # each alone in its block of weights, beside zeros
        w = torch.zeros(130, 384, dtype=torch.bfloat16, device="cuda")
        w[129] = row
        q, s = mbw.quantize_fp8_b128(w)
        want, scale = plain_blocks(w)
        assert same(s, scale) and same(q, want)


def test_norm_of_awkward_rows():
    x, wn = awkward(), torch.linspace(0.5, 2, 384, device="cuda").bfloat16()
    for eps in (1e-6, 0.0):
        r = (1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + eps)).float()
        want, scale = plain_rows((x.float() * r * wn.float()).bfloat16())
        q, s = mbw.quantize_fp8_g128(x, norm_weight=wn, norm_eps=eps)
        assert same(s, scale) and same(q, want)


def test_weights_are_there_for_a_product_queued_behind_them():
    """A product reads weights before it waits for the kernel in front of it; the quantizer ends so that it may."""
    g = gen(9)
    x, xs, _, _ = operands(g, 8, 4, 2048)
    mats = [(torch.randn(2048, 2048, generator=g, device="cuda")).bfloat16() for _ in range(4)]
    torch.cuda.synchronize()
    for w in mats * 3:
        q, s = mbw.quantize_fp8_b128(w)
        got = mbw.gemm_fp8_b128(x, xs, q, s)
        y, mass, eps = exact(x, xs, *plain_blocks(w))
        check(got, y, mass * eps + half_step(y))


def test_compiled_calls_give_the_same_and_refuse_in_the_same_words(monkeypatch):
    from memory_bound_weight_gb300 import _binding as B

    g = gen(11)
    x, xs, w, sc = operands(g, 20, 300, 512)
    wide = torch.randn(20, 600, generator=g, device="cuda").bfloat16()
    wn = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    r = torch.randn(20, 300, generator=g, device="cuda").bfloat16()

    def calls():
        return [*mbw.quantize_fp8_g128(wide[:, 8:520]), *mbw.quantize_fp8_g128(wide[:, :512], norm_weight=wn, norm_eps=1e-5),
                *mbw.quantize_fp8_g128(wide[:1, :512]), *mbw.quantize_fp8_b128(wide[:, :512].contiguous()),
                mbw.dequant_fp8_g128(x, xs), mbw.dequant_fp8_b128(w, sc), mbw.gemm_fp8_b128(x, xs, w, sc),
                mbw.gemm_fp8_b128(x, xs, w, sc, residual=r, up_weights=w, up_scales=sc, workspace=wn)]

    bad = [lambda: mbw.quantize_fp8_g128(wide), lambda: mbw.quantize_fp8_g128(wide[:, :512].float()),
           lambda: mbw.quantize_fp8_g128(wide.t()), lambda: mbw.quantize_fp8_g128(wide[:, :512], norm_weight=wn[:256]),
           lambda: mbw.quantize_fp8_b128(wide[:, :512]), lambda: mbw.dequant_fp8_g128(x, sc), lambda: mbw.dequant_fp8_b128(x, xs),
           lambda: mbw.gemm_fp8_b128(x, xs[:, :3], w, sc), lambda: mbw.gemm_fp8_b128(x, xs, w, sc, residual=r[:, :100]),
           lambda: mbw.gemm_fp8_b128(x, xs, w[:, :256].contiguous(), sc), lambda: mbw.gemm_fp8_b128(x, xs, w, sc, up_weights=w),
           lambda: mbw.gemm_fp8_b128(x, xs, w, sc, up_weights=w[:100].contiguous(), up_scales=sc),
           lambda: mbw.gemm_fp8_b128(x, xs, w, sc, workspace=torch.zeros(4)), lambda: mbw.gemm_fp8_b128(x.cpu(), xs, w, sc)]

    def said():
        out = []
        for f in bad:
            with pytest.raises((TypeError, ValueError)) as e:
                f()
            out.append((e.type, str(e.value)))
        return out

    fast, words = calls(), said()
    assert B._fast and B._fast.gemm_fp8(x, xs, w, sc, None, None, None, None) is not None
    with monkeypatch.context() as m:
        m.setattr(B, "_fast", False)
        slow, slow_words = calls(), said()
    assert words == slow_words
    for a, b in zip(fast, slow):
        assert a.dtype == b.dtype and a.shape == b.shape and same(a, b)
    mbw.inject_launch_failures(1)
    with pytest.raises(mbw.MbwError):
        mbw.gemm_fp8_b128(x, xs, w, sc)
    with mbw.output_fp32():
        assert mbw.gemm_fp8_b128(x, xs, w, sc).dtype == torch.float32


def test_a_first_call_may_be_a_captured_one():
    """In a process of its own: nothing that a call does once, for a kernel or a device, is refused while a stream is captured."""
    code = """
import torch, memory_bound_weight_gb300 as mbw
g = torch.Generator(device="cuda").manual_seed(1)
x, w = (torch.randn(300, 512, generator=g, device="cuda").bfloat16() for _ in range(2))
B, hk, D, pages = 64, 2, 64, 1024
cache = mbw.Kv4Cache(torch.zeros(pages + B, mbw.kv4_page_bytes(16, hk, D, 32), dtype=torch.uint8, device="cuda"), hk, D, 16, 32)
b = torch.arange(B, dtype=torch.int32, device="cuda")
table = torch.cat((torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1), pages + b[:, None]), 1)
q, ctx = torch.randn(B, 16, D, generator=g, device="cuda").bfloat16(), pages * 16 + 1 + b % 16
ws = mbw.kv4_attention_shared_workspace(D, B, 16)
def run():
    wq, sw = mbw.quantize_fp8_b128(w)
    out = []
    for m in (1, 12, 40, 100, 300):
        xq, sx = mbw.quantize_fp8_g128(x[:m])
        out += [mbw.gemm_fp8_b128(xq, sx, wq, sw), mbw.gemm_fp8_b128(xq, sx, wq, sw, up_weights=wq, up_scales=sw)]
    return out + [mbw.kv4_attention_shared(cache, q, table, ctx, pages * 16, workspace=ws)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
mbw.check_device_error()
print("the same")
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "the same" in done.stdout, done.stderr[-2000:]


def test_norm_of_many_rows():
    """Rows by warps, whose sums begin with a power of two above their squares: the codes of the exact mean, in any order of columns."""
    g = gen(12)
    for k in (128, 1280, 3584, 4096):
        x = torch.randn(1300, k, generator=g, device="cuda")
        x[:300] *= torch.exp(4 * torch.randn(300, k, generator=g, device="cuda"))
        x[300:400, 1:] *= 2.0 ** -30
        x[400:500] = x[400:500].abs().sort(1).values  # what is added grows
        x[500:510] *= 2.0 ** -50  # squares near the end of fp32's range, and past it
        x[510:520] *= 2.0 ** 55
        x[520:530] *= 2.0 ** -70
        x[530] = 0
        x = x.bfloat16()
        wn = (1 + 0.3 * torch.randn(k, generator=g, device="cuda")).bfloat16()
        for eps in (1e-6, 0.0):
            r = (1 / torch.sqrt(x.double().square().mean(1, keepdim=True) + eps)).float()
            want, scale = plain_rows((x.float() * r * wn.float()).bfloat16())
            q, s = mbw.quantize_fp8_g128(x, norm_weight=wn, norm_eps=eps)
            assert same(s, scale) and same(q, want)
