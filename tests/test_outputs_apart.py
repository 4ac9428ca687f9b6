"""Outputs and workspaces that share memory with an input are refused; operands that only lie
between each other's rows and columns are not."""
import ctypes

import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16, FP32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu
INV = exm.ERR_INVALID_ARGUMENT

# addresses far apart from each other, never dereferenced
X, W, Y, OFF, RI, WS, DY = (i << 40 for i in range(1, 8))


def mm(x=X, ldx=64, x_rows=8, ri=None, off=OFF, w=W, ldw=64, wst=64 * 32, rows=8, N=32, K=64, E=2, out=0, y=Y, ldy=32, ws=None,
       wsb=0):
    return exm._lib.exmoe_grouped_mm(x, ldx, x_rows, ri, 1, off, w, ldw, wst, rows, N, K, E, 0, out, y, ldy, ws, wsb, None)


def dgrad(dy=DY, lddy=32, off=OFF, w=W, ldw=64, wst=64 * 32, f2s=None, k=1, rows=8, N=32, K=64, E=2, out=0, dx=X, lddx=64,
          ws=None, wsb=0):
    return exm._lib.exmoe_grouped_mm_dgrad(dy, lddy, off, w, ldw, wst, f2s, k, rows, N, K, E, 0, out, dx, lddx, ws, wsb, None)


def wgrad(dy=DY, lddy=32, x=X, ldx=64, x_rows=8, ri=None, off=OFF, rows=8, N=32, K=64, E=2, out=2, dw=W, lddw=64,
          dwst=64 * 32, ws=None, wsb=0):
    return exm._lib.exmoe_grouped_mm_wgrad(dy, lddy, x, ldx, x_rows, ri, 1, off, rows, N, K, E, 0, out, dw, lddw, dwst, ws,
                                           wsb, None)


A, B, RANKS, SCALES, IDS = (i << 40 for i in range(8, 13))


def lora(x=X, ldx=64, w=W, ids=IDS, T=4, N=64, K=64, y=Y, ldy=64, ws=WS, **kw):
    f = dict(a=A, lda=64, a_stride=64 * 16, b=B, ldb=16, b_stride=64 * 16, ranks=RANKS, scales=SCALES, adapters=3, rank_max=16)
    f.update(kw)
    return exm._lib.exmoe_lora_linear(x, ldx, w, 64, ctypes.byref(exm.LoraBankC(**f)), ids, T, N, K, 0, y, ldy, ws, 1 << 20,
                                      None)


def refused(status, *names):
    assert status == INV, (status, exm.last_error())
    assert exm.last_error() == "%s overlaps %s" % names


def test_forward_product():
    refused(mm(y=X), "y", "x")
    refused(mm(y=W + 2 * (64 * 64 - 1)), "y", "w")             # the last element of the last expert
    refused(mm(y=W - 2 * (7 * 32 + 31)), "y", "w")             # the last element of y
    refused(mm(y=OFF + 8, out=2), "y", "expert_offsets")
    refused(mm(ri=Y + 4 * 7), "y", "row_index")
    refused(mm(x_rows=100, ri=RI, y=X + 2 * 64 * 99), "y", "x")          # all of x's rows count
    refused(mm(x=X, ldx=96, y=X + 2 * 63, ldy=96), "y", "x")             # columns of one matrix, one of them shared
    refused(mm(x=X + 2 * 31, ldx=96, y=X, ldy=96), "y", "x")
    refused(mm(x=X, ldx=128, y=X + 2 * 64, ldy=48), "y", "x")            # rows of y run into the next row of x
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_MM, 512, 32, 63, 2)
    far = dict(x_rows=512, rows=512, K=63, wsb=need)
    refused(mm(ws=Y - need + 16, **far), "workspace", "y")
    refused(mm(ws=X, **far), "workspace", "x")
    refused(mm(ws=W, **far), "workspace", "w")
    refused(mm(ws=OFF, **far), "workspace", "expert_offsets")


def test_gradient_of_x():
    refused(dgrad(dx=DY), "dx", "dy")
    refused(dgrad(dx=W + 128), "dx", "w")
    refused(dgrad(off=X + 2 * 64 * 8 - 4), "dx", "expert_offsets")
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_DGRAD, 8, 32, 64, 2, 2)
    refused(dgrad(f2s=X + 4, k=2, ws=WS, wsb=need), "dx", "flat_to_sorted")
    refused(dgrad(f2s=RI, k=2, ws=DY, wsb=need), "workspace", "dy")
    refused(dgrad(f2s=RI, k=2, ws=RI - need + 16, wsb=need), "workspace", "flat_to_sorted")
    refused(dgrad(f2s=RI, k=2, ws=X, wsb=need), "workspace", "dx")


def test_gradient_of_w():
    refused(wgrad(dw=X), "dw", "x")
    refused(wgrad(dw=DY - 4), "dw", "dy")
    refused(wgrad(dw=DY - 4 * (2 * 64 * 32) + 4), "dw", "dy")
    refused(wgrad(dw=DY - 4 * (64 * 33), dwst=64 * 33), "dw", "dy")      # into the second expert's first row
    refused(wgrad(ri=W + 16), "dw", "row_index")
    refused(wgrad(off=W), "dw", "expert_offsets")
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_WGRAD, 1 << 16, 32, 64, 2, 0)
    refused(wgrad(rows=1 << 16, x_rows=1 << 16, ws=X + 1024, wsb=need), "workspace", "x")


def test_adapters():
    refused(lora(y=X), "y", "x")
    refused(lora(y=X, w=None), "y", "x")
    refused(lora(y=W), "y", "w")
    refused(lora(y=A + 2 * 64 * 16 * 3 - 2), "y", "bank->a")
    refused(lora(y=A + (1 << 30), a_stride=1 << 29), "y", "bank->a")
    refused(lora(y=B), "y", "bank->b")
    refused(lora(ids=Y), "y", "adapter_ids")
    refused(lora(ranks=Y + 4 * 126), "y", "bank->ranks")
    refused(lora(scales=Y), "y", "bank->scales")
    refused(lora(ws=Y), "workspace", "y")
    refused(lora(ws=X), "workspace", "x")
    refused(lora(ws=B + 64), "workspace", "bank->b")
    refused(lora(ws=IDS), "workspace", "adapter_ids")


@gpu
def test_the_same_tensor_twice():
    x = torch.ones((40, 64), dtype=BF16, device="cuda")
    w, off = torch.ones((2, 64, 64), dtype=BF16, device="cuda"), torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    bank = exm.LoraBank(torch.ones((3, 8, 64), dtype=BF16, device="cuda"), torch.ones((3, 64, 8), dtype=BF16, device="cuda"))
    ids = torch.zeros(40, dtype=torch.int32, device="cuda")
    for call in (lambda: exm.grouped_mm(x, w, off, y=x), lambda: exm.grouped_mm_dgrad(x, w, off, dx=x),
                 lambda: exm.grouped_mm_wgrad(w.view(-1, 64)[:40], x, off, out_dtype=BF16, dw=w),
                 lambda: exm.lora_linear(x, None, bank, ids, y=x), lambda: exm.lora_linear(x, w[0], bank, ids, y=x)):
        with pytest.raises(RuntimeError, match="overlaps"):
            call()
    assert bool((x == 1).all())


def whole(gen, shape):
    return torch.randint(-2, 3, shape, generator=gen).double()


@gpu
@pytest.mark.parametrize("rows", [12, 300])
def test_between_each_others_rows_and_columns(rows):
    """x and y as columns of one buffer, y before x, y in the gaps between x's rows at twice their
    distance, y right behind x, a gradient between the weights' rows: all allowed, all right."""
    gen = torch.Generator().manual_seed(rows)
    N, K, E = 40, 72, 3
    x, w, dy = whole(gen, (rows, K)), whole(gen, (E, N, K)), whole(gen, (rows, N))
    off = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32)
    ref = torch.zeros((rows, N), dtype=torch.float64)
    for e in range(E):
        ref[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w[e].t()
    offd, wd = off.cuda(), w.to(BF16).cuda()

    def check(xd, yd):
        xd.copy_(x)
        exm.grouped_mm(xd, wd, offd, y=yd)
        assert torch.equal(yd.cpu(), ref.to(BF16)) and torch.equal(xd.cpu().double(), x)

    buf = torch.zeros((rows, K + N), dtype=BF16, device="cuda")
    check(buf[:, :K], buf[:, K:])
    check(buf[:, N:], buf[:, :N])
    buf = torch.zeros((2 * rows, K + N), dtype=BF16, device="cuda")
    check(buf[:rows, :K], buf[::2, K:])
    flat = torch.zeros(rows * (K + N), dtype=BF16, device="cuda")
    check(flat[:rows * K].view(rows, K), flat[rows * K:].view(rows, N))
    check(flat[rows * N:].view(rows, K), flat[:rows * N].view(rows, N))
    wide = torch.zeros((E, N, 2 * K), dtype=BF16, device="cuda")          # weights and their gradient side by side
    wide[..., :K].copy_(w)
    dyd, xd = dy.to(BF16).cuda(), x.to(BF16).cuda()
    exm.grouped_mm_wgrad(dyd, xd, offd, out_dtype=BF16, dw=wide[..., K:])
    dw = torch.stack([dy[off[e]:off[e + 1]].t() @ x[off[e]:off[e + 1]] for e in range(E)])
    assert torch.equal(wide[..., K:].cpu(), dw.to(BF16)) and torch.equal(wide[..., :K].cpu().double(), w)
    # the adapters' output beside their input
    L, R = 2, 8
    a, b = whole(gen, (L, R, K)).sign(), whole(gen, (L, N, R)).sign()
    ids = torch.arange(rows) % L
    buf = torch.zeros((rows, K + N + 8), dtype=BF16, device="cuda")
    buf[:, :K].copy_(x)
    bank = exm.LoraBank(a.to(BF16).cuda(), b.to(BF16).cuda())
    exm.lora_linear(buf[:, :K], None, bank, ids.to(torch.int32).cuda(), y=buf[:, K:K + N])
    want = torch.stack([b[int(i)] @ (a[int(i)] @ x[t]) for t, i in enumerate(ids)])
    assert torch.equal(buf[:, K:K + N].cpu(), want.to(BF16))
