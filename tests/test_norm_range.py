"""The norm of rows whose squares leave the range of 32 bits, and of small ones with a small eps: y is of order one
there (or h / sqrt(eps)), as the formula gives in 64 bits. Tolerance: NORM_DELTA (its derivation stands in
test_fp8_experts.py; the row's scaling is by a power of two, eps's by two more roundings), half a step of the type, and
below the normal values of 32 bits the roundings of h r and of (h r) w, each by half of 2^-149, the first of them times
|w| < 3: 2^-148."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

from test_fp8_codes import wrong  # noqa: E402
from test_fp8_experts import BF16, FP16, FP32, NORM_DELTA, norm_ref  # noqa: E402

gpu = pytest.mark.gpu
DELTA = NORM_DELTA + 2.0 ** -23
SIZES = [1e-45, 1e-40, 1e-38, 1e-30, 1e-25, 1e-20, 1e-13, 1e-11, 1e13, 1e15, 1e17, 1e19, 1e25, 1e30, 1e37, 3e38]


def rows(H, dtype):
    """One row of each size, of normal values up to it; then the same with one value alone, and a row of zeros."""
    gen = torch.Generator().manual_seed(H)
    v = torch.randn((len(SIZES), H), generator=gen, dtype=torch.float64)
    v = v / v.abs().amax(1, keepdim=True) * torch.tensor(SIZES, dtype=torch.float64)[:, None]
    one = torch.zeros_like(v)
    one[:, H // 2] = v[:, H // 2].sign() * torch.tensor(SIZES, dtype=torch.float64)
    return torch.cat([v, one, torch.zeros((1, H), dtype=torch.float64)]).to(dtype)


def check(x, w, eps, residual=None, label=""):
    h, ref = norm_ref(x, w, eps, residual)
    zero = (h == 0).all(1)
    o = exm.rms_norm(x.cuda(), w.cuda(), eps, residual=None if residual is None else residual.cuda(), out="both")
    y, bound = o.y.cpu().double(), DELTA * ref.abs() + 2.0 ** -148
    if x.dtype is not FP32:
        fi = torch.finfo(x.dtype)
        bound = bound + fi.eps / 2 * (ref.abs() + bound).clamp(min=fi.tiny)
    bad = ~((y - ref).abs() <= bound)
    if eps == 0:
        assert bool(torch.isnan(y[zero]).all()), label           # (0 / 0)
        bad[zero] = False
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:4].tolist()}"
    if eps == 0 and x.dtype is FP32:                             # (the others' small rows are coarse, y is of order one)
        assert wrong(ref[~zero], o.q[~zero.cuda()], o.scale[~zero.cuda()], DELTA) == (0, 0), label


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [1, 100, 512, 1003, 2048, 4096, 6000, 16384])
def test_rows_of_any_size(H, dtype):
    x, gen = rows(H, dtype), torch.Generator().manual_seed(H + 1)
    w = (1 + 0.2 * torch.randn(H, generator=gen)).to(dtype)
    for eps in torch.tensor([0.0, 1e-40, 1e-30, 1e-12, 1e-6, 1e20, 3e38]).tolist():      # (as 32 bits hold them)
        check(x, w, eps, label=f"eps {eps}")
    check(x / 2, w, 0.0, residual=x / 2, label="residual")
    check((x / 2).to(dtype), w, float(torch.tensor(1e-30)), residual=(x / 4).float(), label="residual in 32 bits")


@gpu
def test_small_rows_in_fp16():
    x = torch.tensor([[6e-8, 0.0, -6e-8, 1.2e-7], [65504.0, -65504.0, 1.0, 0.0]]).to(FP16)
    check(x, torch.ones(4, dtype=FP16), 0.0)
