"""The router's balance and z losses and their gradient against 64 bits.

Tolerances. A softmax in fp32: l - max is rounded once (2^-24 of at most 2^5 here), its exponential is
off by 2^-22, the sum of E <= 256 of them by 2^-20 at most, the quotient by 2^-23: a relative DELTA of
2^-18 for p, and an absolute one of 2^-18 for the log-sum-exp (and 2^-23 of it). Sums over tokens run
over at most 64 terms a lane before they go on pairwise: 2^-18 more."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
gpu = pytest.mark.gpu
INV, UNS = exm.ERR_INVALID_ARGUMENT, exm.ERR_UNSUPPORTED
DELTA = 2.0 ** -18
L, IDS, MASK, LOSS, CNT, WSP, GRAD, DL = (i << 40 for i in range(1, 9))


def fwd(l=L, ldl=8, ids=IDS, mask=None, T=40, E=8, k=2, dt=0, losses=LOSS, counts=CNT, ws=WSP, wsb=1 << 20):
    return exm._lib.exmoe_balance_loss(exm._BALANCE.pack(*(v or 0 for v in (l, ldl, ids, mask, losses, counts, 0, 0, 0)), T, E, k, dt, 0),
                                       ws, wsb, None)


def bwd(l=L, ldl=8, counts=CNT, mask=None, grad=GRAD, T=40, E=8, k=2, dt=0, od=0, dl=DL, lddl=8):
    return exm._lib.exmoe_balance_loss_backward(
        exm._BALANCE.pack(*(v or 0 for v in (l, ldl, 0, mask, 0, counts, grad, dl, lddl)), T, E, k, dt, od), None)


def test_refusals():
    for call in (fwd, bwd):
        for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(dt=3), dict(l=None),
                    dict(l=L + 1), dict(ldl=7), dict(counts=None), dict(counts=CNT + 2)):
            assert call(**bad) == INV, bad
        assert call(E=100, k=65, ldl=100, **({"lddl": 100} if call is bwd else {})) == UNS
    for bad in (dict(ids=None), dict(ids=IDS + 1), dict(losses=None), dict(losses=LOSS + 2), dict(ws=WSP + 8)):
        assert fwd(**bad) == INV, bad
    for bad in (dict(ws=None), dict(wsb=8)):
        assert fwd(**bad) == exm.ERR_WORKSPACE
    for bad in (dict(grad=None), dict(grad=GRAD + 1), dict(dl=None), dict(lddl=7), dict(od=1), dict(dl=DL + 1)):
        assert bwd(**bad) == INV, bad
    assert bwd(T=0, l=None, dl=None) == 0
    assert exm.balance_loss_workspace_bytes(-1, 8) == 0 == exm.balance_loss_workspace_bytes(5, 300)


def test_operands_that_share_memory_are_refused():
    def refused(status, *names):
        assert status == INV and exm.last_error() == "%s overlaps %s" % names, exm.last_error()

    refused(fwd(losses=L + 8), "losses", "logits")
    refused(fwd(losses=CNT + 32), "losses", "counts")
    refused(fwd(counts=IDS), "counts", "topk_ids")
    refused(fwd(mask=CNT + 3), "counts", "mask")
    refused(fwd(ws=L), "workspace", "logits")
    refused(fwd(ws=LOSS - 16), "workspace", "losses")
    refused(bwd(dl=L + 2), "dlogits", "logits")
    refused(bwd(dl=L, od=2), "dlogits", "logits")
    refused(bwd(dl=L, lddl=9), "dlogits", "logits")
    refused(bwd(dl=GRAD), "dlogits", "grad_losses")
    refused(bwd(counts=DL + 8), "dlogits", "counts")
    refused(bwd(mask=DL + 8), "dlogits", "mask")


def test_a_tensor_that_asks_for_a_gradient_is_refused():
    l, g = torch.ones((4, 8)), torch.ones(2)
    ids, c = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    for t, call in ((l, lambda: exm.balance_loss(l, ids)), (l, lambda: exm.balance_loss_backward(l, c, 2, g)),
                    (g, lambda: exm.balance_loss_backward(l, c, 2, g))):
        t.requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call()
        t.requires_grad_(False)


@gpu
def test_refusals_of_the_binding():
    l, g = torch.ones((4, 8), device="cuda"), torch.ones(2, device="cuda")
    ids, c = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    for call in (lambda: exm.balance_loss(l.t(), ids), lambda: exm.balance_loss(l, ids[:3]), lambda: exm.balance_loss(l, ids.long()),
                 lambda: exm.balance_loss(l, ids, mask=g), lambda: exm.balance_loss(l, ids, mask=ids[:3, 0] > 0),
                 lambda: exm.balance_loss(l, ids, losses=c), lambda: exm.balance_loss(l, ids, counts=c[:8]),
                 lambda: exm.balance_loss_backward(l, c[:8], 2, g), lambda: exm.balance_loss_backward(l, c, 2, g[:1]),
                 lambda: exm.balance_loss_backward(l, c, 2, g, dlogits=l[:3]), lambda: exm.balance_loss(l.cpu(), ids)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ plain form, 64 bits
def plain(l, ids, mask, E, k):
    """Counts, the two losses as functions of l (64 bits, differentiable), probabilities, lse."""
    live = torch.ones(l.shape[0], dtype=torch.bool) if mask is None else mask.bool()
    M = int(live.sum())
    counts = torch.tensor([int((ids[live] == e).sum()) for e in range(E)] + [M])
    some = live & (l > -float("inf")).any(1)
    rows = l[some]
    lse = torch.logsumexp(rows, 1)
    p = torch.exp(rows - lse[:, None])
    zero = (l[:0] * 0).sum()
    balance = E * (counts[:E].double() / (M * k) * p.sum(0) / M).sum() if M else zero
    z = (lse ** 2).sum() / M if M else zero
    return counts, balance, z, p, lse, some


def inputs(gen, T, E, k, dtype, sigma=2.0):
    l = (torch.randn((T, E), generator=gen) * sigma + torch.randn(E, generator=gen)).to(dtype)
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32) if T else torch.zeros((0, k), dtype=torch.int32)
    return l, ids


def check(l, ids, mask, k, out_dtype=None, label="", ld=0):
    T, E = l.shape
    l64 = l.double().requires_grad_()
    counts, balance, z, p, lse, some = plain(l64, ids, mask, E, k)
    ga, gz = 0.7, -0.3
    (ga * balance + gz * z).backward()
    ld_ = torch.full((T, E + ld), float("nan"), dtype=l.dtype, device="cuda")[:, ld // 2:ld // 2 + E]
    ld_.copy_(l)
    md = None if mask is None else mask.cuda()
    losses, got = exm.balance_loss(ld_, ids.cuda(), md)
    assert torch.equal(got.cpu().long(), counts), label
    M = max(int(counts[E]), 1)
    balance, z, lse = balance.detach(), z.detach(), lse.detach()
    tol_b = 2 * DELTA * float(balance)
    tol_z = 2 * DELTA * float((lse ** 2 + 2 * lse.abs()).sum() / M) + 2.0 ** -30
    assert abs(float(losses[0]) - float(balance)) <= tol_b, (label, float(losses[0]), float(balance))
    assert abs(float(losses[1]) - float(z)) <= tol_z, (label, float(losses[1]), float(z))
    grad = torch.tensor([ga, gz], device="cuda")
    d = exm.balance_loss_backward(ld_, got, k, grad, md, out_dtype=out_dtype)
    assert d.dtype is (out_dtype or l.dtype)
    ref = l64.grad
    f = counts[:E].double() / (M * k)
    bound = torch.zeros((T, E), dtype=torch.float64)
    lse_d, p_d = lse, p.detach()
    bound[some] = 4 * DELTA * p_d / M * (ga * E * (f + (p_d @ f)[:, None]) + 2 * abs(gz) * (lse_d.abs()[:, None] + 1))
    bound += 2.0 ** -126
    if d.dtype != FP32:
        fi = torch.finfo(d.dtype)
        bound = bound + fi.eps / 2 * (ref.abs() + bound).clamp(min=fi.tiny)
    bad = ~((d.cpu().double() - ref).abs() <= bound)
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} of {bad.numel()} gradients off, first {bad.nonzero()[:4].tolist()}"
    return losses, got, d


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 64, 8), (129, 13, 2), (300, 16, 4), (257, 33, 3), (2000, 64, 8), (512, 64, 8), (513, 64, 8),
                                   (1025, 128, 8), (513, 200, 1), (700, 256, 64)])
def test_losses_and_gradient(T, E, k, dtype):
    gen = torch.Generator().manual_seed(T + E)
    l, ids = inputs(gen, T, E, k, dtype)
    check(l, ids, None, k, label="all")
    check(l, ids, torch.rand(T, generator=gen) < 0.6, k, out_dtype=FP32, label="masked")
    check(l, ids, None, k, label="strided", ld=3)


@gpu
def test_long_batches():
    gen = torch.Generator().manual_seed(1)
    l, ids = inputs(gen, 1000, 64, 6, FP32)
    l, ids = l.repeat(70, 1) + torch.randn((70000, 1), generator=gen), ids.repeat(70, 1)
    check(l, ids, torch.arange(70000) % 7 != 3, 6)


@gpu
def test_masks_that_leave_nothing():
    gen = torch.Generator().manual_seed(2)
    l, ids = inputs(gen, 50, 8, 2, BF16)
    l[::2] = float("nan")                   # masked rows hold anything
    ids[::2] = 1 << 20
    mask = torch.arange(50) % 2 == 1
    losses, counts, d = check(torch.where(mask[:, None], l, torch.zeros_like(l)), ids, mask, 2)
    md, grad = mask.cuda(), torch.tensor([0.7, -0.3], device="cuda")
    losses2, counts2 = exm.balance_loss(l.cuda(), ids.cuda(), md)
    assert torch.equal(losses, losses2) and torch.equal(counts, counts2)
    d2 = exm.balance_loss_backward(l.cuda(), counts2, 2, grad, md)
    assert torch.equal(d, d2) and bool((d2[::2] == 0).all())
    none = torch.zeros(50, dtype=torch.bool, device="cuda")
    losses, counts = exm.balance_loss(l.cuda(), ids.cuda(), none)
    assert losses.tolist() == [0, 0] and counts.tolist() == [0] * 9
    assert bool((exm.balance_loss_backward(l.cuda(), counts, 2, grad, none) == 0).all())
    losses, counts = exm.balance_loss(l[:0].cuda(), ids[:0].cuda())
    assert losses.tolist() == [0, 0] and counts.tolist() == [0] * 9
    assert exm.balance_loss_backward(l[:0].cuda(), counts, 2, grad).shape == (0, 8)


@gpu
def test_infinite_logits_and_ids_outside():
    gen = torch.Generator().manual_seed(3)
    l, ids = inputs(gen, 60, 24, 3, FP32)
    l[4, :23] = -float("inf")               # one expert left
    l[5, 3], l[6, 20:] = -float("inf"), torch.finfo(FP32).min
    l[7] = -float("inf")                    # none left: counts, adds nothing
    ids[9, 1], ids[10, 0] = -1, 24
    l64 = l.double()
    counts, balance, z, p, lse, some = plain(l64, ids, None, 24, 3)
    assert not bool(some[7]) and int(counts.sum()) == 60 + 60 * 3 - 2
    losses, got = exm.balance_loss(l.cuda(), ids.cuda())
    assert torch.equal(got.cpu().long(), counts)
    assert abs(float(losses[0] - balance)) <= 2 * DELTA * float(balance) and abs(float(losses[1] - z)) <= 2 * DELTA * float((lse ** 2 + 2 * lse.abs()).sum()) / 60
    d = exm.balance_loss_backward(l.cuda(), got, 3, torch.tensor([1.0, 1.0], device="cuda")).cpu()
    assert bool((d[7] == 0).all()) and bool(torch.isfinite(d).all()) and float(d[5, 3]) == 0 and bool((d[4, :23] == 0).all())
    l[8, 2] = float("nan")
    losses, got = exm.balance_loss(l.cuda(), ids.cuda())
    d = exm.balance_loss_backward(l.cuda(), got, 3, torch.tensor([1.0, 1.0], device="cuda")).cpu()
    assert bool(torch.isnan(losses).all()) and bool(torch.isnan(d[8]).all()) and bool(torch.isfinite(d[[i for i in range(60) if i != 8]]).all())


@gpu
def test_gradient_against_differences():
    """(f(l + s v) - f(l - s v)) / 2 s of the kernel's own losses along random v, s = 2^-4: the third
    derivative's part is s^2 / 6 |f'''| |v|^3, below 2^-8 of |v|; the losses' own error 2 DELTA f / s."""
    gen = torch.Generator().manual_seed(4)
    T, E, k = 6, 12, 3
    l, ids = inputs(gen, T, E, k, FP32, sigma=1.0)
    _, counts = exm.balance_loss(l.cuda(), ids.cuda())
    s = 2.0 ** -4
    for which in range(2):
        grad = torch.zeros(2)
        grad[which] = 1.0
        d = exm.balance_loss_backward(l.cuda(), counts, k, grad.cuda()).cpu().double()
        for _ in range(5):
            v = torch.randn((T, E), generator=gen)
            v /= v.norm()
            hi, lo = (exm.balance_loss((l + t * v).cuda(), ids.cuda())[0][which].double().cpu() for t in (s, -s))
            f = float(hi + lo) / 2
            assert abs(float((hi - lo) / (2 * s)) - float((d * v.double()).sum())) <= 2.0 ** -8 + 2 * DELTA * f / s


@gpu
def test_in_place_and_given_outputs():
    gen = torch.Generator().manual_seed(5)
    l, ids = inputs(gen, 333, 40, 4, BF16)
    ld, grad = l.cuda(), torch.tensor([0.5, 0.1], device="cuda")
    losses, counts = torch.full((2,), -1.0, device="cuda"), torch.full((41,), -1, dtype=torch.int32, device="cuda")
    ws = torch.full((exm.balance_loss_workspace_bytes(333, 40),), 255, dtype=torch.uint8, device="cuda")
    a, b = exm.balance_loss(ld, ids.cuda(), losses=losses, counts=counts, workspace=ws)
    assert a is losses and b is counts
    want = exm.balance_loss_backward(ld, counts, 4, grad)
    assert exm.balance_loss_backward(ld, counts, 4, grad, dlogits=ld) is ld and torch.equal(ld, want)


@gpu
def test_inside_an_autograd_function_and_a_graph():
    """A router's loss as a user joins the calls: logits from a weight, gradient through it; captured
    and replayed with other inputs."""
    gen = torch.Generator().manual_seed(6)
    T, H, E, k = 100, 64, 16, 2

    class Losses(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids):
            losses, counts = exm.balance_loss(logits, ids)
            ctx.save_for_backward(logits, counts)
            ctx.k = ids.shape[1]
            return losses

        @staticmethod
        def backward(ctx, grad):
            logits, counts = ctx.saved_tensors
            return exm.balance_loss_backward(logits, counts, ctx.k, grad.contiguous()), None

    x, w = torch.randn((T, H), generator=gen), torch.randn((E, H), generator=gen) * 0.1
    ids = inputs(gen, T, E, k, FP32)[1]
    wd = w.cuda().requires_grad_()
    (Losses.apply(x.cuda() @ wd.t(), ids.cuda()) * torch.tensor([1.0, 0.01], device="cuda")).sum().backward()
    w64 = w.double().requires_grad_()
    _, balance, z, _, _, _ = plain(x.double() @ w64.t(), ids, None, E, k)
    (balance + 0.01 * z).backward()
    # (logits in fp32: off by 64 roundings of 2^-24 of their terms, far under a hundredth of a percent)
    assert float((wd.grad.cpu().double() - w64.grad).norm() / w64.grad.norm()) < 1e-4

    l, idd, grad = (x @ w.t()).cuda(), ids.cuda(), torch.tensor([0.3, 0.2], device="cuda")
    losses, counts, d = torch.empty(2, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty((T, E), device="cuda")
    ws = exm.alloc_workspace(exm.balance_loss_workspace_bytes(T, E))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        exm.balance_loss(l, idd, losses=losses, counts=counts, workspace=ws)
        exm.balance_loss_backward(l, counts, k, grad, dlogits=d)
    for i in range(4):
        l.copy_(torch.randn((T, E), generator=gen))
        idd.copy_(inputs(gen, T, E, k, FP32)[1])
        graph.replay()
        torch.cuda.synchronize()
        want, c = exm.balance_loss(l, idd)
        assert torch.equal(losses, want) and torch.equal(counts, c)
        assert torch.equal(d, exm.balance_loss_backward(l, c, k, grad))
