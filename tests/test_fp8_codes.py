"""Every 8-bit value that the quantisers and the norm write, compared so that a NaN counts as wrong, and the
largest values of a group, whose quotient by the scale lies at the border of what e4m3 holds.

Tolerances: those of test_fp8_experts.py (half a step of e4m3, and 2^-21 of the quotient's roundings)."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

from test_fp8_experts import (DTYPES, F8, FP32, NORM_DELTA, SIZES, close, groups_of, norm_ref, on_gpu, randn, spread,  # noqa: E402
                              swiglu_delta)

gpu = pytest.mark.gpu


def wrong(v, q, scale, delta, rows=1, weight=None):
    """How many scales and how many values of q are not those of v (64 bits, known to a relative delta)."""
    q, scale = q.detach().cpu().to(FP32).double(), scale.detach().cpu().double()
    want = (groups_of(v, rows).abs().amax((-3, -1)) / 448).clamp(min=2.0 ** -126)
    w = torch.ones_like(want) if weight is None else weight.double()[:, None].expand_as(want)
    assert scale.shape == want.shape and q.shape == v.shape
    fine = (scale - want * w).abs() <= (delta + 2.0 ** -23) * want * w.abs()
    t = v / spread(want, v.shape[-2], v.shape[-1], rows)
    right = (q - t).abs() <= torch.clamp(2.0 ** -4 * t.abs(), min=2.0 ** -10) + (2 * delta + 2.0 ** -21) * t.abs()
    return int((~fine).sum()), int((~right).sum())


def test_a_nan_counts_as_wrong():
    v = randn(torch.Generator().manual_seed(1), 3, 200).double()
    scale = groups_of(v).abs().amax((-3, -1)) / 448
    q = (v / spread(scale, 3, 200)).float().to(F8)
    assert wrong(v, q, scale, 2.0 ** -23) == (0, 0)
    for bad in (float("nan"), 3 * float(q[1, 7].float()) + 1):
        one = q.float()
        one[1, 7] = bad
        assert wrong(v, one.to(F8), scale, 2.0 ** -23) == (0, 1)
    scale[2, 1] = float("nan")
    assert wrong(v, q, scale, 2.0 ** -23) == (1, 0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 67, 300])
def test_rows(rows, dtype):
    gen = torch.Generator().manual_seed(100 + rows)
    for K in SIZES:
        for shift, more in ((0, 0), (1, 3)):
            x = (randn(gen, rows, K) * torch.exp(2 * randn(gen, rows, 1))).to(dtype)
            assert wrong(x.double(), *exm.quantize_fp8(on_gpu(x, shift, more)), 0.0) == (0, 0), (rows, K, shift)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_largest_value_of_a_group_is_448(dtype):
    """v / scale of the largest |v| is 448 but for three roundings of 2^-24, and e4m3 rounds all below 464 to
    it: for any significand and any power of two, from the least scale on to the type's largest value."""
    gen = torch.Generator().manual_seed(5)
    fi = torch.finfo(dtype)
    lo = max(-116.0, float(torch.tensor(fi.tiny).log2()))
    hi = float(torch.tensor(fi.max, dtype=FP32).log2()) - 1
    top = (1 + torch.rand((20000, 1), generator=gen)) * torch.exp2((torch.rand((20000, 1), generator=gen) * (hi - lo) + lo).floor())
    top = torch.cat([top, torch.tensor([[fi.max], [1.0], [2.0 - 2 * fi.eps], [448.0], [447.9]])]).to(dtype)
    x = top.expand(-1, 136).contiguous()
    x[:, 1::2] *= -1
    x[:, 5] = 0
    q, scale = exm.quantize_fp8(x.cuda())
    want = torch.full(x.shape, 448.0)
    want[:, 1::2] *= -1
    want[:, 5] = 0
    assert torch.equal(q.float().cpu(), want)
    assert wrong(x.double(), q, scale, 0.0) == (0, 0)
    q, scale = exm.quantize_fp8_weights(x[None].cuda().contiguous())
    assert wrong(x[None].double(), q, scale, 0.0, rows=128) == (0, 0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,I", [(1, 1), (3, 127), (130, 200), (257, 1024)])
def test_gate_and_up(rows, I, dtype):
    gen = torch.Generator().manual_seed(200 + rows + I)
    x = randn(gen, rows, 2 * I, sigma=2.0).to(dtype)
    g, u = x.double().split(I, 1)
    h = g / (1 + torch.exp(-g)) * u
    weights = torch.rand(rows, generator=gen)
    xd = on_gpu(x, 1, 5)
    assert wrong(h, *exm.swiglu_fp8(xd), swiglu_delta(g)) == (0, 0)
    assert wrong(h, *exm.swiglu_fp8(xd, weights.cuda()), swiglu_delta(g) + 2.0 ** -24, weight=weights) == (0, 0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (3, 100, 300), (2, 257, 129), (5, 384, 1008)])
def test_weights(E, N, K, dtype):
    gen = torch.Generator().manual_seed(300 + E + N + K)
    w = (randn(gen, E, N, K, sigma=0.02) * torch.exp(randn(gen, E, N, 1))).to(dtype)
    for shift, more in ((0, 0), (3, 1)):
        assert wrong(w.double(), *exm.quantize_fp8_weights(on_gpu(w, shift, more)), 0.0, rows=128) == (0, 0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 100, 512, 1003, 2048, 2056, 4096, 6000, 16384])
def test_norm(H, dtype):
    gen = torch.Generator().manual_seed(400 + H)
    x, w, res = randn(gen, 9, H, sigma=2.0).to(dtype), (1 + randn(gen, H, sigma=0.2)).to(dtype), randn(gen, 9, H, sigma=3.0).to(dtype)
    for r in (None, res):
        _, ref = norm_ref(x, w, 1e-5, r)
        o = exm.rms_norm(on_gpu(x, 1, 1), w.cuda(), 1e-5, residual=None if r is None else r.cuda(), out="both")
        close(o.y, ref, NORM_DELTA, f"{H}")
        assert wrong(ref, o.q, o.scale, NORM_DELTA) == (0, 0), (H, r is None)
