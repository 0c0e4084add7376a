"""Refusals of the 4-bit cache and token calls, in the C ABI and in the
binding, and the rotary tables: no GPU is needed and nothing is launched."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import memory_bound_weight_gb300 as mbw  # noqa: E402
from memory_bound_weight_gb300 import _binding as B  # noqa: E402
from memory_bound_weight_gb300 import build as mbuild  # noqa: E402
from memory_bound_weight_gb300.rope import rope_frequencies  # noqa: E402

P = [0x10000 * (i + 1) for i in range(8)]  # fake aligned addresses: never dereferenced on these paths
INVALID, MISALIGNED, SHAPE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return B.lib()


def cache(pages=P[0], num=4, page=16, heads=2, dim=128, group=64):
    return ctypes.byref(B.MbwKv4Cache(pages, num, page, heads, dim, group))


def rope(cs=P[5], max_pos=10, dim=128, inter=0, pos=P[6]):
    return ctypes.byref(B.MbwRope(cs, max_pos, dim, inter, pos))


BAD_CACHES = [(dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(page=2048), SHAPE), (dict(page=0), SHAPE),
              (dict(page=-16), SHAPE), (dict(dim=96), SHAPE), (dict(dim=512), SHAPE), (dict(group=128), SHAPE),
              (dict(group=0), SHAPE), (dict(heads=0), SHAPE), (dict(heads=2000), SHAPE), (dict(num=0), INVALID),
              (dict(num=-1), INVALID), (dict(num=1 << 31), SHAPE), (dict(pages=None), INVALID),
              (dict(pages=P[0] + 8), MISALIGNED)]


def append(L, c=None, k=P[1], ks=256, v=P[2], vs=256, slots=P[3], q=P[4], qs=512, qo=P[4], os=512, hq=4, r=None, T=3):
    return L.mbw_kv4_append(c or cache(), k, ks, v, vs, slots, q, qs, qo, os, hq, r, T, None)


def attend(L, c=None, q=P[1], qs=512, out=P[2], os=512, lse=None, table=P[3], ts=4, tw=4, ctx=P[4], starts=None, b=2,
           T=2, hq=4, scale=0.1, window=0, ws=None, wn=0):
    return L.mbw_kv4_attention(c or cache(), q, qs, out, os, lse, table, ts, tw, ctx, starts, b, T, hq, scale, window,
                               ws, wn, None)


def logprobs(L, x=P[0], fp32=0, stride=100, t=P[1], M=3, V=100, scale=1.0, k=2, ws=None):
    return L.mbw_token_logprobs(x, fp32, stride, t, M, V, scale, k, P[2], P[3], P[4], P[5], P[6], ws, 0, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_is_checked_by_every_call(L, change, status):
    c = cache(**change)
    assert append(L, c) == status
    assert L.mbw_kv4_gather(c, P[1], P[2], P[3], 3, None) == status
    assert attend(L, c) == status
    assert L.mbw_last_error().decode().startswith("mbw_kv4_attention: ")


def test_no_cache_at_all(L):
    assert L.mbw_kv4_append(None, P[1], 256, P[2], 256, P[3], None, 0, None, 0, 0, None, 1, None) == INVALID
    assert L.mbw_kv4_gather(None, P[1], P[2], P[3], 3, None) == INVALID
    assert L.mbw_kv4_attention(None, P[1], 512, P[2], 512, None, P[3], 4, 4, P[4], None, 2, 2, 4, 0.1, 0, None, 0,
                               None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(hq=-1), INVALID), (dict(T=1 << 31), SHAPE), (dict(hq=70000, qs=1 << 24, os=1 << 24), SHAPE),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(q=None), INVALID),
    (dict(qo=None), INVALID), (dict(ks=248), SHAPE), (dict(vs=255), SHAPE), (dict(qs=504), SHAPE), (dict(os=0), SHAPE),
    (dict(k=P[1] + 2), MISALIGNED), (dict(v=P[2] + 8), MISALIGNED), (dict(q=P[4] + 4), MISALIGNED),
    (dict(qo=P[4] + 8), MISALIGNED), (dict(slots=P[3] + 4), MISALIGNED), (dict(ks=260), MISALIGNED),
    (dict(os=514), MISALIGNED), (dict(T=0), 0),
])
def test_append_refuses(L, change, status):
    assert append(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(cs=None), INVALID), (dict(pos=None), INVALID), (dict(max_pos=0), INVALID), (dict(inter=2), INVALID),
    (dict(dim=0), SHAPE), (dict(dim=8), SHAPE), (dict(dim=24), SHAPE), (dict(dim=144), SHAPE),
    (dict(cs=P[5] + 8), MISALIGNED), (dict(pos=P[6] + 2), MISALIGNED),
])
def test_append_refuses_rotations(L, change, status):
    assert append(L, r=rope(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(b=-1), INVALID), (dict(window=-1), INVALID), (dict(tw=-1), INVALID),
    (dict(hq=3), SHAPE), (dict(hq=0), SHAPE), (dict(T=3), SHAPE), (dict(b=0), INVALID), (dict(b=(1 << 20) + 1), SHAPE),
    (dict(T=1 << 30, b=1 << 10), SHAPE), (dict(tw=1 << 28, ts=1 << 28), SHAPE), (dict(ts=3), SHAPE),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ctx=None), INVALID), (dict(table=None), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(qs=504), SHAPE), (dict(os=500), SHAPE),
    (dict(q=P[1] + 2), MISALIGNED), (dict(out=P[2] + 8), MISALIGNED), (dict(table=P[3] + 2), MISALIGNED),
    (dict(ctx=P[4] + 1), MISALIGNED), (dict(starts=P[5] + 2), MISALIGNED), (dict(lse=P[6] + 2), MISALIGNED),
    (dict(ws=P[7] + 4, wn=64), MISALIGNED), (dict(qs=516), MISALIGNED), (dict(T=0), 0), (dict(T=0, b=0), 0),
])
def test_attention_refuses(L, change, status):
    assert attend(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(k=-1), INVALID), (dict(fp32=2), INVALID),
    (dict(M=1 << 31), SHAPE), (dict(V=1 << 31, stride=1 << 31), SHAPE), (dict(k=33), SHAPE), (dict(V=0), SHAPE),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(stride=99), SHAPE), (dict(x=None), INVALID), (dict(x=P[0] + 1), MISALIGNED),
    (dict(x=P[0] + 2, fp32=1), MISALIGNED), (dict(t=P[1] + 2), MISALIGNED), (dict(ws=P[7] + 8), MISALIGNED),
    (dict(M=0), 0),
])
def test_logprobs_refuses(L, change, status):
    assert logprobs(L, **change) == status


def test_sizes(L):
    for page in (16, 48, 1024):
        for dim in (64, 128, 256):
            for group in (32, 64):
                assert L.mbw_kv4_page_bytes(page, 3, dim, group) == mbw.kv4_page_bytes(page, 3, dim, group) == \
                    3 * page * (dim + 8 * dim // group)
    assert L.mbw_kv4_page_bytes(8, 3, 64, 32) == 0
    for bad in ((8, 1, 64, 32), (16, 0, 64, 32), (16, 1, 80, 32), (16, 1, 64, 16)):
        with pytest.raises(ValueError):
            mbw.kv4_page_bytes(*bad)
    assert L.mbw_kv4_attention_workspace_bytes(96) == 0
    assert L.mbw_status_string(8).decode() == "MBW_ERR_DEVICE_RANGE"


# ----------------------------------------------------------------- binding ----
class Host(torch.Tensor):
    """A host tensor that says it is a CUDA tensor."""

    @property
    def is_cuda(self):
        return True


def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Host)


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append((name, len(a))) or 0

    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(B, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(B, "_device_index", lambda: -1)  # a host tensor's
    return made


def host_cache(page=16, heads=2, dim=128, group=64):
    return mbw.Kv4Cache(host(3, mbw.kv4_page_bytes(page, heads, dim, group), dtype=torch.uint8), heads, dim, page, group)


def test_valid_calls_marshal(calls):
    c, i32, i64 = host_cache(), torch.int32, torch.int64
    wide = host(5, 8, 128)
    q, k, v = wide[:, :4], wide[:, 4:6], wide[:, 6:]
    assert mbw.kv4_append(c, k, v, host(5, dtype=i64)) is None
    out = mbw.kv4_append(c, k, v, host(5, dtype=i64), q=q, positions=host(5, dtype=i32),
                         cos_sin=host(9, 64, dtype=torch.float32), interleaved=True)
    assert out.shape == (5, 4, 128) and mbw.kv4_append(c, k, v, host(5, dtype=i64), q=q, q_out=q) is q
    assert mbw.kv4_gather(c, host(7, dtype=i64))[1].shape == (7, 2, 128)
    assert mbw.kv4_attention(c, q, host(5, 3, dtype=i32), host(5, dtype=i32)).shape == (5, 4, 128)
    o, lse = mbw.kv4_attention(c, q, host(2, 3, dtype=i32), host(2, dtype=i32), host(3, dtype=i32), out=q, window=5,
                               return_lse=True, workspace=host(64, dtype=torch.uint8))
    assert o is q and lse.shape == (5, 4)
    r = mbw.token_logprobs(host(3, 50)[:, 1:], host(3, dtype=i32), top_k=4)
    assert r.top_ids.shape == (3, 4) and r.rank.shape == (3,)
    assert mbw.token_logprobs(host(3, 50, dtype=torch.float32)).logprob is None
    for name, n in calls:
        assert n == len(B.SIGNATURES[name][0]), name
    assert len(calls) == 8


def test_bad_tensors_never_reach_the_library(calls):
    c, i32, i64, f32 = host_cache(), torch.int32, torch.int64, torch.float32
    q, k, s = host(5, 4, 128), host(5, 2, 128), host(5, dtype=i64)
    bad = [
        (lambda: mbw.Kv4Cache(host(3, 100, dtype=torch.uint8), 2, 128), ValueError, "bytes per page"),
        (lambda: mbw.Kv4Cache(torch.zeros(3, 4608, dtype=torch.uint8), 2, 128), ValueError, "CUDA tensor"),
        (lambda: mbw.kv4_append(c, host(5, 3, 128), k, s), ValueError, "k must have shape"),
        (lambda: mbw.kv4_append(c, k, host(4, 2, 128), s), ValueError, "same number"),
        (lambda: mbw.kv4_append(c, k, host(5, 2, 128, dtype=f32), s), TypeError, "v must be"),
        (lambda: mbw.kv4_append(c, k, host(5, 128, 2).transpose(1, 2), s), ValueError, "contiguous rows"),
        (lambda: mbw.kv4_append(c, torch.zeros(5, 2, 128).bfloat16(), k, s), ValueError, "CUDA tensor"),
        (lambda: mbw.kv4_append(c, k, k, host(5, dtype=i32)), TypeError, "slots"),
        (lambda: mbw.kv4_append(c, k, k, host(4, dtype=i64)), ValueError, "slots"),
        (lambda: mbw.kv4_append(c, k, k, s, q=host(4, 4, 128)), ValueError, "q and k"),
        (lambda: mbw.kv4_append(c, k, k, s, q_out=q), ValueError, "q_out without q"),
        (lambda: mbw.kv4_append(c, k, k, s, q=q, q_out=host(5, 2, 128)), ValueError, "q_out"),
        (lambda: mbw.kv4_append(c, k, k, s, positions=host(5, dtype=i32)), ValueError, "together"),
        (lambda: mbw.kv4_append(c, k, k, s, positions=host(5, dtype=i64), cos_sin=host(9, 64, dtype=f32)), TypeError,
         "positions"),
        (lambda: mbw.kv4_append(c, k, k, s, positions=host(5, dtype=i32), cos_sin=host(9, 64)), TypeError, "cos_sin"),
        (lambda: mbw.kv4_gather(c, host(5, dtype=i32)), TypeError, "slots"),
        (lambda: mbw.kv4_attention(c, host(5, 4, 64), host(5, 3, dtype=i32), host(5, dtype=i32)), ValueError, "q must"),
        (lambda: mbw.kv4_attention(c, q, host(5, 3, dtype=i64), host(5, dtype=i32)), TypeError, "block_table"),
        (lambda: mbw.kv4_attention(c, q, host(5, 3, dtype=i32), host(4, dtype=i32)), ValueError, "ctx_lens"),
        (lambda: mbw.kv4_attention(c, q, host(5, 3, dtype=i32), host(5, dtype=i32), host(5, dtype=i32)), ValueError,
         "q_starts"),
        (lambda: mbw.kv4_attention(c, q, host(5, 3, dtype=i32), host(5, dtype=i32), out=host(4, 4, 128)), ValueError, "out"),
        (lambda: mbw.token_logprobs(torch.zeros(3, 5)), ValueError, "CUDA tensor"),
        (lambda: mbw.token_logprobs(host(3, 5, dtype=torch.float16)), TypeError, "logits"),
        (lambda: mbw.token_logprobs(host(5, 3).T), ValueError, "contiguous rows"),
        (lambda: mbw.token_logprobs(host(3, 5), host(2, dtype=i32)), ValueError, "targets"),
        (lambda: mbw.token_logprobs(host(3, 5), top_k=33), ValueError, "top_k"),
    ]
    for call, err, words in bad:
        with pytest.raises(err, match=words):
            call()
    assert calls == []


# ------------------------------------------------------------------ tables ----
def test_rope_table_is_the_formula():
    t = mbw.rope_table(300, 32, 1e4, device="cpu")
    assert t.shape == (300, 32) and t.dtype == torch.float32
    for p in (0, 1, 299):
        for i in (0, 7, 15):
            a = p * 1e4 ** (-2 * i / 32)
            assert abs(t[p, i].item() - math.cos(a)) < 2.0 ** -24 and abs(t[p, 16 + i].item() - math.sin(a)) < 2.0 ** -24


def test_rope_scalings():
    plain, one = rope_frequencies(64, 1e4)
    assert one == 1.0
    lin, _ = rope_frequencies(64, 1e4, {"type": "linear", "factor": 4})
    assert torch.equal(lin, plain / 4)
    ntk, _ = rope_frequencies(64, 1e4, {"type": "ntk", "factor": 8})
    assert ntk[0] == 1 and abs(ntk[-1] * 8 / plain[-1] - 1) < 1e-12  # the slowest pair turns 8 times slower
    yarn, times = rope_frequencies(64, 1e4, {"type": "yarn", "factor": 16, "original_max": 4096})
    turns = 4096 * plain / (2 * math.pi)
    assert abs(times - (0.1 * math.log(16) + 1)) < 1e-15
    assert torch.equal(yarn[turns > 40], plain[turns > 40]) and torch.allclose(yarn[turns < 0.7], plain[turns < 0.7] / 16)
    assert ((yarn <= plain) & (yarn >= plain / 16 * (1 - 1e-12))).all() and (yarn[1:] < yarn[:-1]).all()
    l3, _ = rope_frequencies(128, 5e5, {"type": "llama3", "factor": 8, "original_max": 8192, "low_freq_factor": 1,
                                        "high_freq_factor": 4})
    base, _ = rope_frequencies(128, 5e5)
    turns = 8192 * base / (2 * math.pi)
    for f, g, n in zip(l3.tolist(), base.tolist(), turns.tolist()):
        k = min(1.0, max(0.0, (n - 1) / 3))
        assert abs(f - (g * k + g / 8 * (1 - k))) < 1e-15


@pytest.mark.parametrize("args", [(0, 32), (10, 24), (10, 0), (10, 32, 1.0), (10, 32, 1e4, {"type": "other"}),
                                  (10, 32, 1e4, {"type": "linear", "factor": 0.5}),
                                  (10, 32, 1e4, {"type": "linear", "factr": 2})])
def test_rope_table_refuses(args):
    with pytest.raises(ValueError):
        mbw.rope_table(*args, device="cpu")
