"""One adapter or one expert: the distance to the next one means nothing, whatever it is."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16 = torch.bfloat16
gpu = pytest.mark.gpu


def whole(gen, shape):
    return torch.randint(-2, 3, shape, generator=gen).double()


def first_of(t, width):
    """t [1, R, C] as the first entry of a tensor whose entries are `width` elements apart."""
    store = torch.full((2, width), float("nan"), dtype=BF16, device="cuda")
    view = store.as_strided(t.shape, (width, t.shape[2], 1))
    view.copy_(t)
    assert view.stride(0) == width and view.data_ptr() % 16 == 0
    return view


@gpu
@pytest.mark.parametrize("T", [1, 40, 200])
def test_one_adapter(T):
    gen = torch.Generator().manual_seed(T)
    N, K, R = 48, 64, 16
    x, w, a, b = whole(gen, (T, K)), whole(gen, (N, K)), whole(gen, (1, R, K)).sign(), whole(gen, (1, N, R)).sign()
    bank = exm.LoraBank(first_of(a, R * K + 5), first_of(b, N * R + 3))
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    y = exm.lora_linear(x.to(BF16).cuda(), w.to(BF16).cuda(), bank, ids)
    assert torch.equal(y.cpu(), (x @ w.t() + (x @ a[0].t()) @ b[0].t()).to(BF16))


@gpu
@pytest.mark.parametrize("rows", [3, 300])
def test_one_expert(rows):
    gen = torch.Generator().manual_seed(rows)
    N, K = 48, 64
    x, w, dy = whole(gen, (rows, K)), whole(gen, (1, N, K)), whole(gen, (rows, N))
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    xd, dyd, wd = x.to(BF16).cuda(), dy.to(BF16).cuda(), first_of(w, N * K + 5)
    assert torch.equal(exm.grouped_mm(xd, wd, off).cpu(), (x @ w[0].t()).to(BF16))
    assert torch.equal(exm.grouped_mm_dgrad(dyd, wd, off).cpu(), (dy @ w[0]).to(BF16))
    dw = first_of(torch.zeros_like(w), N * K + 3)
    exm.grouped_mm_wgrad(dyd, xd, off, out_dtype=BF16, dw=dw)
    assert torch.equal(dw.cpu(), (dy.t() @ x).unsqueeze(0).to(BF16))


def test_one_adapter_any_stride():
    """Past the stride check (the workspace is missing): no stride of a single adapter is refused."""
    import ctypes
    far = [i << 40 for i in range(1, 7)]
    for stride in (0, 7, 64 * 16 + 4):
        bank = exm.LoraBankC(far[0], 64, stride, far[1], 16, stride, None, None, 1, 16)
        st = exm._lib.exmoe_lora_linear(far[2], 64, None, 0, ctypes.byref(bank), far[3], 4, 32, 64, 0, far[4], 32, None, 0, None)
        assert st == exm.ERR_WORKSPACE, (stride, exm.last_error())
