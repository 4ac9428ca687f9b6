"""Rows quantised as they are with a routing weight in their scales (tolerances: test_fp8_experts.py)."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

from test_fp8_codes import wrong  # noqa: E402
from test_fp8_experts import DTYPES, on_gpu, randn  # noqa: E402

gpu = pytest.mark.gpu


def test_weights_that_ask_for_a_gradient_are_refused():
    with pytest.raises(ValueError, match="gradient"):
        exm.quantize_fp8(torch.ones((4, 256)), weights=torch.ones(4, requires_grad=True))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 127), (130, 200), (257, 1024)])
def test_rows_and_their_weights(rows, K, dtype):
    gen = torch.Generator().manual_seed(rows + K)
    x = randn(gen, rows, K, sigma=2.0).to(dtype)
    xd = on_gpu(x, 1, 5)
    q, scale = exm.quantize_fp8(xd)
    weights = torch.rand((rows + 3) * 2, generator=gen)
    index = torch.randint(0, len(weights), (rows,), generator=gen).to(torch.int32)
    index[rows // 2] = -1 if rows % 2 else len(weights)          # no weight: zeros
    w = torch.where((index >= 0) & (index < len(weights)), weights[index.clamp(0, len(weights) - 1).long()], torch.tensor(0.0))
    for weight, got in ((w, exm.quantize_fp8(xd, weights=weights.cuda(), row_index=index.cuda())), (weights[:rows], exm.quantize_fp8(xd, weights=weights.cuda()))):
        assert torch.equal(got[0].float(), q.float()) and torch.equal(got[1], scale * weight.cuda()[:, None])
        assert wrong(x.double(), *got, 2.0 ** -24, weight=weight) == (0, 0)
    for bad in (dict(weights=weights.double().cuda()), dict(weights=weights), dict(weights=weights.cuda(), row_index=index.cuda()[1:]),
                dict(weights=weights.cuda(), row_index=index.long().cuda())):
        with pytest.raises(ValueError):
            exm.quantize_fp8(xd, **bad)
    for bad in (dict(row_index=index.cuda()), dict(weights=weights[:rows - 1].cuda()) if rows > 1 else dict(row_index=index.cuda())):
        with pytest.raises(RuntimeError):
            exm.quantize_fp8(xd, **bad)
