"""The products and the adapters record no gradient: a tensor that asks for one is refused, unless
gradients are off. (The refusal comes before any look at the device, so it runs on the CPU.)"""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16 = torch.bfloat16
gpu = pytest.mark.gpu


class Bank:
    def __init__(self, dev="cpu"):
        self.a, self.b = torch.ones((2, 8, 64), dtype=BF16, device=dev), torch.ones((2, 32, 8), dtype=BF16, device=dev)


def calls(dev):
    t = dict(x=torch.ones((6, 64), dtype=BF16, device=dev), w=torch.ones((2, 32, 64), dtype=BF16, device=dev),
             dy=torch.ones((6, 32), dtype=BF16, device=dev), y=torch.ones((6, 32), dtype=BF16, device=dev),
             dx=torch.ones((6, 64), dtype=BF16, device=dev), dw=torch.ones((2, 32, 64), dtype=BF16, device=dev),
             w2=torch.ones((32, 64), dtype=BF16, device=dev))
    off, ids = torch.tensor([0, 2, 6], dtype=torch.int32, device=dev), torch.zeros(6, dtype=torch.int32, device=dev)
    bank = Bank(dev)
    t["a"], t["b"] = bank.a, bank.b

    def lora(w):
        use = bank if dev == "cpu" else exm.LoraBank(bank.a, bank.b)
        return exm.lora_linear(t["x"], w, use, ids, y=t["y"])

    return t, [(("x", "w", "y"), lambda: exm.grouped_mm(t["x"], t["w"], off, y=t["y"])),
               (("dy", "w", "dx"), lambda: exm.grouped_mm_dgrad(t["dy"], t["w"], off, dx=t["dx"])),
               (("dy", "x", "dw"), lambda: exm.grouped_mm_wgrad(t["dy"], t["x"], off, out_dtype=BF16, dw=t["dw"])),
               (("x", "w2", "a", "b", "y"), lambda: lora(t["w2"])), (("x", "a", "b", "y"), lambda: lora(None))]


def test_a_tensor_that_asks_for_a_gradient_is_refused():
    t, every = calls("cpu")
    for names, call in every:
        for name in names:
            t[name].requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="GPU"):      # past that refusal
                call()
            t[name].requires_grad_(False)


@gpu
def test_the_same_results_without_recording():
    t, every = calls("cuda")
    for names, call in every:
        t["y"].fill_(1.0)
        want = call().clone()
        for name in names:
            if name in ("y", "dx", "dw"):
                continue
            t[name].requires_grad_()
            t["y"].fill_(1.0)
            with torch.no_grad():
                got = call()
            assert torch.equal(got, want) and not got.requires_grad
            t[name].requires_grad_(False)


@gpu
def test_inside_an_autograd_function():
    """A layer made of the three products, as a user joins them."""
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return exm.grouped_mm(x, w, off)

        @staticmethod
        def backward(ctx, dy):
            x, w = ctx.saved_tensors
            return (exm.grouped_mm_dgrad(dy.contiguous(), w, off),
                    exm.grouped_mm_wgrad(dy.contiguous(), x, off, out_dtype=w.dtype))

    gen = torch.Generator().manual_seed(1)
    x = torch.randint(-2, 3, (6, 64), generator=gen).double()
    w = torch.randint(-2, 3, (2, 32, 64), generator=gen).double()
    xd, wd = x.to(BF16).cuda().requires_grad_(), w.to(BF16).cuda().requires_grad_()
    Product.apply(xd, wd).sum().backward()
    seg = torch.tensor([0, 0, 1, 1, 1, 1])
    assert torch.equal(xd.grad.cpu(), w.sum(1)[seg].to(BF16))
    want = torch.stack([x[:2].sum(0), x[2:].sum(0)]).unsqueeze(1).expand(2, 32, 64)
    assert torch.equal(wd.grad.cpu(), want.to(BF16))
