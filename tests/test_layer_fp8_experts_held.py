"""Tensors that a program put into Fp8Experts itself: the layer refuses what does not fit the experts' sizes, before
a kernel reads it."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("name", ["gate_up", "gate_up_scale", "down", "down_scale"])
def test_each_of_them_is_checked(name):
    T, H, I, E, k = 4, 256, 128, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, wn, wr = randn(T, H).bfloat16(), randn(H).bfloat16(), randn(E, H).bfloat16()
    ex = exm.Fp8Experts(randn(E, 2 * I, H), randn(E, H, I))
    want = exm.moe_layer_fp8(x, wn, wr, ex, k).y
    fits = getattr(ex, name)
    other = torch.float32 if fits.dtype is torch.float8_e4m3fn else torch.bfloat16
    for bad in (fits[:E - 1].contiguous(), fits.transpose(1, 2), fits.to(other), fits.cpu()):
        setattr(ex, name, bad)
        with pytest.raises(ValueError, match="experts." + name):
            exm.moe_layer_fp8(x, wn, wr, ex, k)
    setattr(ex, name, fits.clone().requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        exm.moe_layer_fp8(x, wn, wr, ex, k)
    setattr(ex, name, fits.clone())
    assert torch.equal(exm.moe_layer_fp8(x, wn, wr, ex, k).y, want)
