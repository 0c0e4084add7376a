"""token_logprobs' top tokens where many logits pass for the best: rising rows, ties, masks, and pieces that fill the buffer
of candidates. The order is by logit, then by the lower index, whatever the order in which they are met."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

INF = float("inf")


def rows(kind, M, V):
    g = torch.Generator(device="cuda")
    g.manual_seed(V + M)
    i = torch.arange(V, device="cuda").float().expand(M, V)
    if kind == "rising":
        return i / V * 9 - 4
    if kind == "falling":
        return 5 - i / V * 9
    if kind == "equal":
        return torch.full((M, V), 1.25, device="cuda")
    x = torch.randn(M, V, generator=g, device="cuda") * 2
    if kind == "ties":
        return x.round()
    if kind == "late":  # the first logits, which make the first gate, are masked
        x[:, :V // 2] = -INF
    if kind == "few":   # fewer logits than asked for are not masked
        x[:, torch.randperm(V, generator=g, device="cuda")[:V - 5]] = -INF
    return x


@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "ties", "late", "few"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,k", [(1, 152064, 20), (3, 40001, 32), (50, 30011, 7), (2, 2500, 32), (7, 333, 1), (500, 9000, 20)])
def test_top_tokens(kind, dtype, M, V, k):
    x = rows(kind, M, V).to(dtype)
    order = torch.sort(x.double(), dim=1, descending=True, stable=True)
    lp = x.double().log_softmax(1)
    want = lp.gather(1, order.indices[:, :k])
    for ws in (None, mbw.token_logprobs_workspace()):
        got = mbw.token_logprobs(x, order.indices[:, min(k, V) // 2].int().contiguous(), top_k=k, workspace=ws)
        ids = order.indices[:, :k].int()
        # what is masked has probability 0, in any order after the rest; tokens that there are not are -1
        real = order.values[:, :k] > -INF
        assert torch.equal(got.top_ids[real], ids[real])
        assert (got.top_logprobs[~real] == -INF).all()
        # a term's exponent is off by 2^-22 of it, fp32 sums of them by as much, the result by its own rounding
        assert ((got.top_logprobs.double() - want)[real].abs() <= (1 + want[real].abs()) * 1e-5).all()
        if kind != "few":
            assert (got.rank == min(k, V) // 2 + 1).all()
