"""Refusals of the 8-bit floating point calls and of attention behind a shared
prefix, in the C ABI and in the binding: no GPU is needed and nothing is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import memory_bound_weight_gb300 as mbw  # noqa: E402
from memory_bound_weight_gb300 import _binding as B  # noqa: E402
from memory_bound_weight_gb300 import build as mbuild  # noqa: E402

P = [0x10000 * (i + 1) for i in range(10)]  # fake aligned addresses: never dereferenced on these paths
INVALID, MISALIGNED, SHAPE = 1, 2, 3
MAX = (1 << 31) - (1 << 16)


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return B.lib()


def product(L, x=P[0], xs=P[1], w=P[2], ws=P[3], y=P[4], M=3, N=200, K=256, ws_at=None, ws_n=0, fusion=True, **fuse):
    f = B.MbwFusion()
    for name, value in fuse.items():
        setattr(f, name, value)
    return L.gemm_fp8_b128(x, xs, w, ws, y, M, N, K, ctypes.byref(f) if fusion else None, ws_at, ws_n, None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-128), INVALID), (dict(M=MAX + 1), SHAPE),
    (dict(N=MAX + 1), SHAPE), (dict(K=MAX + 128), SHAPE), (dict(K=0), SHAPE), (dict(K=64), SHAPE), (dict(K=200), SHAPE),
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID),
    (dict(y=None), INVALID), (dict(x=P[0] + 8), MISALIGNED), (dict(xs=P[1] + 2), MISALIGNED),
    (dict(w=P[2] + 16), MISALIGNED), (dict(ws=P[3] + 1), MISALIGNED), (dict(y=P[4] + 2), MISALIGNED),
    (dict(ws_at=P[9] + 8, ws_n=1 << 20), MISALIGNED), (dict(norm_weight=P[5]), INVALID), (dict(up_zeros=P[5]), INVALID),
    (dict(up_weights=P[5]), INVALID), (dict(up_scales=P[6]), INVALID), (dict(up_weights=P[5] + 16, up_scales=P[6]), MISALIGNED),
    (dict(up_weights=P[5], up_scales=P[6] + 2), MISALIGNED), (dict(residual=P[7] + 1), MISALIGNED),
    (dict(M=0), 0), (dict(N=0), 0), (dict(M=0, x=None, xs=None, fusion=False), 0),
])
def test_product_refuses(L, change, status):
    assert product(L, **change) == status
    if status:
        assert L.mbw_last_error().decode().startswith("gemm_fp8_b128: ")


@pytest.mark.parametrize("args,status", [
    ((P[0], 256, P[1], P[2], -1, 256, None, 0.0), INVALID), ((P[0], 256, P[1], P[2], 3, -128, None, 0.0), INVALID),
    ((P[0], 256, P[1], P[2], 3, 0, None, 0.0), SHAPE), ((P[0], 256, P[1], P[2], 3, 250, None, 0.0), SHAPE),
    ((P[0], 248, P[1], P[2], 3, 256, None, 0.0), SHAPE), ((P[0], 260, P[1], P[2], 3, 256, None, 0.0), MISALIGNED),
    ((None, 256, P[1], P[2], 3, 256, None, 0.0), INVALID), ((P[0], 256, None, P[2], 3, 256, None, 0.0), INVALID),
    ((P[0], 256, P[1], None, 3, 256, None, 0.0), INVALID), ((P[0] + 2, 256, P[1], P[2], 3, 256, None, 0.0), MISALIGNED),
    ((P[0], 256, P[1] + 8, P[2], 3, 256, None, 0.0), MISALIGNED), ((P[0], 256, P[1], P[2] + 2, 3, 256, None, 0.0), MISALIGNED),
    ((P[0], 256, P[1], P[2], 3, 256, P[3] + 2, 0.0), MISALIGNED), ((P[0], 256, P[1], P[2], 3, 256, P[3], -1.0), INVALID),
    ((P[0], 256, P[1], P[2], 3, 256, P[3], float("nan")), INVALID), ((P[0], 256, P[1], P[2], 3, 256, P[3], float("inf")), INVALID),
    ((P[0], 256, P[1], P[2], MAX + 1, 256, None, 0.0), SHAPE), ((None, 0, None, None, 0, 256, None, 0.0), 0),
])
def test_quantizing_tokens_refuses(L, args, status):
    assert L.mbw_quantize_fp8_g128(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((P[0], P[1], P[2], -1, 256), INVALID), ((P[0], P[1], P[2], 3, 0), SHAPE), ((P[0], P[1], P[2], 3, 130), SHAPE),
    ((None, P[1], P[2], 3, 256), INVALID), ((P[0], None, P[2], 3, 256), INVALID), ((P[0], P[1], None, 3, 256), INVALID),
    ((P[0] + 8, P[1], P[2], 3, 256), MISALIGNED), ((P[0], P[1] + 8, P[2], 3, 256), MISALIGNED),
    ((P[0], P[1], P[2] + 2, 3, 256), MISALIGNED), ((P[0], P[1], P[2], MAX + 1, 256), SHAPE), ((None, None, None, 0, 256), 0),
])
def test_quantizing_weights_and_back_refuses(L, args, status):
    assert L.mbw_quantize_fp8_b128(*args, None) == status
    out_of_order = (args[0], args[2], args[1], args[3], args[4])  # codes, scales, values
    assert L.mbw_dequant_fp8_b128(*out_of_order, None) == status
    assert L.mbw_dequant_fp8_g128(*out_of_order, None) == status


def cache(pages=P[0], num=4, page=16, heads=2, dim=128, group=64):
    return ctypes.byref(B.MbwKv4Cache(pages, num, page, heads, dim, group))


def attend(L, c=None, q=P[1], qs=512, out=P[2], os=512, lse=None, table=P[3], ts=4, tw=4, ctx=P[4], starts=None, b=2,
           T=2, hq=4, scale=0.1, window=0, shared=32, ws=None, wn=0):
    return L.mbw_kv4_attention_shared(c or cache(), q, qs, out, os, lse, table, ts, tw, ctx, starts, b, T, hq, scale,
                                      window, shared, ws, wn, None)


@pytest.mark.parametrize("change,status", [
    (dict(shared=-1), INVALID), (dict(shared=65), SHAPE), (dict(shared=1 << 40), SHAPE), (dict(b=-1), INVALID),
    (dict(T=-1), INVALID), (dict(window=-1), INVALID), (dict(hq=3), SHAPE), (dict(T=3), SHAPE), (dict(b=0), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(table=None), INVALID), (dict(ctx=None), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(qs=504), SHAPE), (dict(os=0), SHAPE),
    (dict(q=P[1] + 2), MISALIGNED), (dict(ws=P[5] + 4, wn=64), MISALIGNED), (dict(ts=3), SHAPE), (dict(T=0), 0),
    (dict(c=cache(page=24)), SHAPE),
])
def test_shared_attention_refuses(L, change, status):
    assert attend(L, **change) == status
    if status:
        assert L.mbw_last_error().decode().startswith("mbw_kv4_attention_shared: ")


def test_injected_failures_reach_the_new_calls(L):
    for call in (lambda: product(L), lambda: L.mbw_quantize_fp8_g128(P[0], 256, P[1], P[2], 3, 256, None, 0.0, None),
                 lambda: L.mbw_quantize_fp8_b128(P[0], P[1], P[2], 3, 256, None),
                 lambda: L.mbw_dequant_fp8_b128(P[0], P[1], P[2], 3, 256, None), lambda: attend(L)):
        assert L.mbw_inject_launch_failures(1) == 0
        assert call() == 6 and b"injected" in L.mbw_last_error()


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0

        return fn


@pytest.fixture
def host(monkeypatch):
    """The calls' marshalling on host tensors: the CUDA test is bypassed and the library records."""
    rec = Recorder()

    def plain(t, name, dtype, ndim):
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.dim() != ndim or not t.is_contiguous():
            raise ValueError(f"{name} must have {ndim} dimensions and be contiguous")
        return t.shape

    monkeypatch.setattr(B, "_plain", plain)
    monkeypatch.setattr(B, "lib", lambda: rec)
    monkeypatch.setattr(B, "_fast", False)
    monkeypatch.setattr(B, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(B, "_check_devices", lambda *ts: 0)
    monkeypatch.setattr(B, "_need", lambda t, name, dtype, ndim: plain(t, name, dtype, ndim))
    return rec


def operands(M=3, N=200, K=256):
    e = torch.float8_e4m3fn
    return (torch.zeros(M, K, dtype=e), torch.zeros(M, K // 128), torch.zeros(N, K, dtype=e), torch.zeros(2, K // 128))


def test_products_marshal(host):
    x, xs, w, ws = operands()
    y = mbw.gemm_fp8_b128(x, xs, w, ws, residual=torch.zeros(3, 200, dtype=torch.bfloat16), up_weights=w, up_scales=ws)
    assert y.shape == (3, 200) and y.dtype == torch.bfloat16
    assert mbw.gemm_fp8_b128(x[:0], xs[:0], w, ws).shape == (0, 200)
    for name, args in host.calls:
        assert name == "gemm_fp8_b128" and len(args) == len(B.SIGNATURES[name][0])
        assert args[6:8] == (200, 256)
    assert mbw.dequant_fp8_g128(x, xs).shape == (3, 256)
    assert mbw.dequant_fp8_b128(w, ws).shape == (200, 256)
    assert mbw.quantize_fp8_b128(torch.zeros(200, 256, dtype=torch.bfloat16))[1].shape == (2, 2)
    for name, args in host.calls:
        assert len(args) == len(B.SIGNATURES[name][0]), name


@pytest.mark.parametrize("change", [
    dict(x=torch.zeros(3, 256)), dict(x=torch.zeros(3, 250, dtype=torch.float8_e4m3fn)), dict(xs=torch.zeros(3, 3)),
    dict(xs=torch.zeros(2, 3)), dict(xs=torch.zeros(3, 2, dtype=torch.float64)), dict(ws=torch.zeros(200, 2)),
    dict(ws=torch.zeros(1, 2)), dict(w=torch.zeros(200, 384, dtype=torch.float8_e4m3fn)), dict(w=torch.zeros(200, 256, dtype=torch.uint8)),
    dict(residual=torch.zeros(3, 199, dtype=torch.bfloat16)), dict(residual=torch.zeros(3, 200)),
    dict(out=torch.zeros(3, 200)), dict(out=torch.zeros(4, 200, dtype=torch.bfloat16)),
    dict(up_weights=operands()[2]), dict(up_scales=operands()[3]),
    dict(up_weights=torch.zeros(100, 256, dtype=torch.float8_e4m3fn), up_scales=operands()[3]),
    dict(up_weights=operands()[2], up_scales=torch.zeros(2, 1)),
    dict(x=torch.zeros(256, 3, dtype=torch.float8_e4m3fn).t()),
])
def test_products_refuse_in_the_binding(host, change):
    x, xs, w, ws = operands()
    kw = dict(x=x, xs=xs, w=w, ws=ws)
    kw.update(change)
    with pytest.raises((TypeError, ValueError)):
        mbw.gemm_fp8_b128(kw.pop("x"), kw.pop("xs"), kw.pop("w"), kw.pop("ws"), **kw)
    assert host.calls == []


def test_host_tensors_are_refused():
    x, xs, w, ws = operands()
    with pytest.raises(ValueError, match="CUDA tensor"):
        mbw.gemm_fp8_b128(x, xs, w, ws)
    for call in (mbw.quantize_fp8_g128, mbw.quantize_fp8_b128):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(torch.zeros(3, 256, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mbw.quantize_fp8_g128([1.0])


def test_workspaces(L):
    for args in ((96, 4, 4), (128, -1, 4), (128, 4, 0), (128, 1 << 31, 1), (128, 1 << 20, 1 << 16)):
        assert L.mbw_kv4_attention_shared_workspace_bytes(*args) == 0
    for d in (64, 128, 256):
        assert L.mbw_kv4_attention_shared_workspace_bytes(d, 10, 8) >= L.mbw_kv4_attention_workspace_bytes(d)


def test_shared_attention_needs_its_length():
    with pytest.raises(TypeError, match="shared_len"):
        mbw.kv4_attention_shared(None, None, None, None, None)
