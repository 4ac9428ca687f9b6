"""8-bit outputs that ask for a gradient are refused, as other outputs are, and are left as they were."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu


def q8(*shape, device="cpu"):
    return torch.full(shape, 7.0, device=device).to(torch.float8_e4m3fn).requires_grad_()


def test_weights_in_8_bits():
    with pytest.raises(ValueError, match="gradient"):
        exm.quantize_fp8_weights(torch.ones((1, 4, 256)), q=q8(1, 4, 256))


@gpu
def test_rows_in_8_bits():
    x, w = torch.ones((4, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    calls = [(256, lambda q: exm.quantize_fp8(x, q=q)), (128, lambda q: exm.swiglu_fp8(x, q=q)), (256, lambda q: exm.rms_norm(x, w, out="fp8", q=q)),
             (256, lambda q: exm.quantize_fp8_weights(x[None], q=q[None]))]
    for K, call in calls:
        q = q8(4, K, device="cuda")
        with pytest.raises(ValueError, match="gradient"):
            call(q)
        torch.cuda.synchronize()
        assert bool((q.detach().float() == 7).all())
        with torch.no_grad():            # (asked to record none: written)
            call(q)
        assert not bool((q.detach().float() == 7).all())
