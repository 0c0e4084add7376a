"""8-bit operands that begin where the calls allow it and no allocation does: codes of activations on 16 bytes, scales on 4,
weights on 32. Where an operand lies changes no bit of a result."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

import memory_bound_weight_gb300 as mbw  # noqa: E402
from test_fp8_gpu import check, exact, gen, half_step, operands  # noqa: E402


def moved(t, by):
    """A copy that begins `by` bytes behind an allocation's beginning."""
    n = t.numel() * t.element_size()
    buf = torch.empty(n + by, dtype=torch.uint8, device="cuda")
    out = buf[by:].view(t.dtype).view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 256 == by and out.is_contiguous()
    return out


# every kernel of the product, and of that of few rows both widths; 16 rows of small and of large weights
@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (3, 77, 128), (8, 1000, 3584), (9, 640, 1152), (12, 300, 512), (16, 130, 256),
                                   (16, 3584, 18944), (40, 700, 1152), (100, 300, 640), (300, 513, 896)])
def test_activations_on_16_bytes(m, n, k):
    g = gen(m + n)
    x, xs, w, sc = operands(g, m, n, k)
    _, _, u, su = operands(g, 1, n, k)
    y, mass, eps = exact(x, xs, w, sc)
    want, gated = mbw.gemm_fp8_b128(x, xs, w, sc), mbw.gemm_fp8_b128(x, xs, w, sc, up_weights=u, up_scales=su)
    check(want, y, mass * eps + half_step(y))
    for by in (16, 48, 240):
        at = moved(x, by), moved(xs, by - 12), moved(w, 32), moved(sc, 4)
        assert torch.equal(mbw.gemm_fp8_b128(*at), want)
        assert torch.equal(mbw.gemm_fp8_b128(*at, up_weights=moved(u, 32), up_scales=moved(su, 8)), gated)


@pytest.mark.parametrize("m", [3, 1300])
def test_quantizers_on_16_bytes(m):
    g = gen(m)
    x, wn = torch.randn(m, 1152, generator=g, device="cuda").bfloat16(), torch.rand(1152, generator=g, device="cuda").bfloat16()
    for by in (16, 48):
        for norm in (None, wn):
            a, b = mbw.quantize_fp8_g128(x, norm), mbw.quantize_fp8_g128(moved(x, by), None if norm is None else moved(norm, by))
            assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
            assert torch.equal(mbw.dequant_fp8_g128(moved(a[0], by), moved(a[1], 4)), mbw.dequant_fp8_g128(*a))
        a, b = mbw.quantize_fp8_b128(x), mbw.quantize_fp8_b128(moved(x, by))
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
        assert torch.equal(mbw.dequant_fp8_b128(moved(a[0], by), moved(a[1], 4)), mbw.dequant_fp8_b128(*a))
