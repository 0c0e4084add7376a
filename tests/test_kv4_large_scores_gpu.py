"""kv4_attention with scores of any size, up to where softmax is the largest key alone.

A score is off by what its roundings move: fp32 sums, and in chunks also s (n - 8) rounded to fp16. An output is then a mean
of the values of the keys that can have a weight: those within twice that, and 40 (e^-40 of a weight), of the largest."""
import pytest
import torch

import kv4_ref as ref
import memory_bound_weight_gb300 as mbw
from test_kv4_chunk_gpu import cache_of, starts_of
from test_kv4_gpu import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [-1e20, 1.0, 1e3, 3e4, 1e6, 1e7, 1e9, 1e12, 1e20])
@pytest.mark.parametrize("ctx,nq,hq,hk,d,group", [
    ([600, 40], [1, 1], 8, 2, 128, 64), ([90, 700, 5], [2, 5, 3], 6, 2, 64, 32), ([300], [4], 4, 1, 256, 64),
    ([300], [60], 8, 2, 256, 64), ([400, 150], [140, 150], 16, 2, 128, 64), ([500], [300], 8, 2, 64, 32),
])
def test_scores_of_any_size(ctx, nq, hq, hk, d, group, scale):
    cache, table, kv, g = cache_of(95, ctx, 16, hk, d, group, lambda g, n: (normal(g, n, hk, d), normal(g, n, hk, d)))
    starts = starts_of(nq)
    q = normal(g, starts[-1], hq, d)
    c, s = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ctx, starts))
    x = ref.f64(q)
    for ws in (None, mbw.kv4_attention_workspace(d)):
        out, lse = (ref.f64(t) for t in mbw.kv4_attention(cache, q, table, c, s, scale=scale, return_lse=True, workspace=ws))
        assert out.isfinite().all() and lse.isfinite().all()
        for b, ((kn, ks, km), (vn, vs, vm)) in enumerate(kv):
            for h in range(hq):
                i = h * hk // hq
                k, v = kn[:, i] * ks[:, i] + km[:, i], vn[:, i] * vs[:, i] + vm[:, i]
                kc = (ks[:, i] * (kn[:, i] - 8)).abs()
                for t in range(starts[b], starts[b + 1]):
                    n = ctx[b] - nq[b] + t - starts[b] + 1
                    y = k[:n] @ x[t, h] * scale
                    off = float((x[t, h].abs() @ (kc[:n] * 2.0 ** -11 + k[:n].abs() * 2.0 ** -18).T).max()) * abs(scale)
                    can = v[:n][y >= y.max() - 2 * off - 40]
                    room = v[:n].abs().amax(0) * (2.0 ** -8 + 2.0 ** -9)  # bf16's rounding, and that of the weights
                    assert (out[t, h] >= can.amin(0) - room).all() and (out[t, h] <= can.amax(0) + room).all()
                    want = torch.logsumexp(y, 0)
                    assert abs(lse[t, h] - want) <= off + 2.0 ** -9 + abs(want) * 2.0 ** -22
