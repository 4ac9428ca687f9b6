"""A shared projection beside low-rank adapters of many requests (lora_linear) against a
plain fp64 form, token by token.

Tolerance of one output. Products of 16-bit values are exact in fp32; a sum of R of them is
off by at most R 2^-23 S, S the sum of absolute products. So v is off by ev = K 2^-23 |A||x|.
The two 16-bit halves of v (scaled so that the token's largest is in [1, 2)) hold it to half
a step of half a step, 2^-8 2^-8 of it (bf16) or 2^-11 2^-11 of it, in fp16 at least 2^-25 of
the largest: eh = 2^-16 |v|, or 2^-22 |v| + 2^-25 max |v|. Their products with B are exact and summed over 2 rank
terms. Altogether
  K 2^-23 |W||x| + |scale| (|B| (ev + eh) + 2 rank 2^-23 |B||v|) + 3 2^-23 |y parts|,
the last for the two fp32 roundings of scaling and adding. The 16-bit output adds half a
step, eps / 2 of its value (at least eps / 2 of the smallest normal number). Without W, y is
read exactly. Small whole numbers come out equal bit for bit."""
import ctypes

import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

FAKE = 0x10000
BF16, FP16 = torch.bfloat16, torch.float16
gpu = pytest.mark.gpu


def plain(x, w, a, b, ids, ranks, scales, y0=None):
    """fp64 on the CPU: result and the bound above (without the output's rounding)."""
    T, K = x.shape
    N = b.shape[1]
    y = torch.zeros((T, N), dtype=torch.float64) if y0 is None else y0.clone()
    bound = torch.zeros_like(y)
    if w is not None:
        y = x @ w.t()
        bound = x.abs() @ w.abs().t() * K * 2.0 ** -23
    parts = y.abs()
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < a.shape[0]:
            continue
        r, s = int(ranks[i]), float(scales[i])
        if r == 0:
            continue
        A, B = a[i, :r], b[i, :, :r]
        v = A @ x[t]
        ev = (A.abs() @ x[t].abs()) * K * 2.0 ** -23
        eh = 2.0 ** -16 * v.abs() + 2.0 ** -25 * v.abs().max()
        y[t] += s * (B @ v)
        bound[t] += abs(s) * (B.abs() @ (ev + eh) + 2 * r * 2.0 ** -23 * (B.abs() @ v.abs()))
        parts[t] = parts[t] + abs(s) * (B @ v).abs()
    return y, bound + 3 * 2.0 ** -23 * parts


def close(got, ref, bound, label):
    # a reference that overflows the output type, or that an infinite weight makes infinite,
    # has to come out infinite or NaN (inf - inf of the two halves of v): there is no distance
    fi = torch.finfo(got.dtype)
    got64, finite = got.detach().cpu().double(), ref.isfinite() & (ref.abs() + bound < fi.max)
    assert not bool(got64[~ref.isfinite()].isfinite().any()), f"{label}: finite where the formula is not"
    bound = bound + fi.eps / 2 * (ref.abs() + bound).clamp(min=fi.tiny)
    bad = ~((got64 - ref).abs() <= bound) & finite
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} outside the bound, first {bad.nonzero()[:4].tolist()}"


def normal(gen, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=gen) * sigma).to(dtype).double()


def whole(gen, shape, lo=-2, hi=3):
    return torch.randint(lo, hi, shape, generator=gen).double()


# ------------------------------------------------------------------ refusals (no GPU)
def _call(x=FAKE, ldx=64, w=FAKE, ldw=64, ids=FAKE, T=4, N=32, K=64, dt=0, y=FAKE, ldy=32, ws=FAKE, wsb=1 << 20, bank=True,
          **kw):
    f = dict(a=FAKE, lda=64, a_stride=64 * 16, b=FAKE, ldb=16, b_stride=32 * 16, ranks=None, scales=None, adapters=3,
             rank_max=16)
    f.update(kw)
    b = exm.LoraBankC(**f)
    return exm._lib.exmoe_lora_linear(x, ldx, w, ldw, ctypes.byref(b) if bank else None, ids, T, N, K, dt, y, ldy, ws,
                                      wsb, None)


def test_refusals():
    inv = exm.ERR_INVALID_ARGUMENT
    for bad in (dict(bank=False), dict(T=-1), dict(N=0), dict(K=0), dict(K=60), dict(K=4), dict(adapters=0),
                dict(rank_max=0), dict(rank_max=12), dict(rank_max=136), dict(dt=2), dict(x=None), dict(x=FAKE + 8),
                dict(ldx=56), dict(ldx=68), dict(w=FAKE + 2), dict(ldw=32), dict(a=None), dict(lda=32), dict(b=None),
                dict(ldb=8), dict(a_stride=64 * 16 - 8), dict(b_stride=32 * 16 - 8), dict(a_stride=64 * 16 + 4),
                dict(y=None), dict(y=FAKE + 1), dict(ldy=31), dict(ids=None), dict(ids=FAKE + 2), dict(ranks=FAKE + 1),
                dict(scales=FAKE + 2), dict(ws=FAKE + 4)):
        assert _call(**bad) == inv, bad
        assert exm.last_error() != ""
    need = exm.lora_workspace_bytes(4, 32, 64, 3, 16)
    assert need > 0
    assert _call(wsb=need - 1) == exm.ERR_WORKSPACE and str(need) in exm.last_error()
    assert _call(ws=None) == exm.ERR_WORKSPACE
    assert _call(T=0) == exm.OK
    for far in (dict(ldx=(1 << 24) + 8), dict(ldw=(1 << 24) + 8), dict(lda=(1 << 24) + 8, a_stride=1 << 30)):
        assert _call(**far) == exm.ERR_UNSUPPORTED, far
    assert _call(T=1 << 22, N=1 << 20, ldy=1 << 20, b_stride=1 << 24) == exm.ERR_UNSUPPORTED
    assert exm.lora_workspace_bytes(4, 32, 60, 3, 16) == 0


def test_binding_refuses_cpu_tensors():
    a, b = torch.zeros(2, 8, 16, dtype=BF16), torch.zeros(2, 5, 8, dtype=BF16)
    with pytest.raises(ValueError, match="GPU"):
        exm.LoraBank(a, b)


# ------------------------------------------------------------------ GPU
def device_bank(a, b, ranks, scales, dtype):
    return exm.LoraBank(a.to(dtype).cuda(), b.to(dtype).cuda(), ranks=ranks.to(torch.int32).cuda(),
                        scales=scales.float().cuda())


@gpu
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 40, 129, 300])
@pytest.mark.parametrize("N,K,L,R", [(64, 64, 1, 8), (130, 200, 5, 24), (257, 8, 40, 128), (3, 520, 7, 64)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_against_fp64(T, N, K, L, R, dtype):
    print(f"lora T={T} N={N} K={K} L={L} R={R} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(T * 1009 + N)
    x, w = normal(gen, (T, K), dtype), normal(gen, (N, K), dtype, 0.1)
    a, b = normal(gen, (L, R, K), dtype, 0.1), normal(gen, (L, N, R), dtype, 0.1)
    ranks = torch.randint(0, R + 1, (L,), generator=gen)
    ranks[0] = R
    scales = torch.rand(L, generator=gen) * 3 - 1
    ids = torch.randint(-1, L, (T,), generator=gen)
    bank = device_bank(a, b, ranks, scales, dtype)
    xd, wd, idd = x.to(dtype).cuda(), w.to(dtype).cuda(), ids.to(torch.int32).cuda()
    close(exm.lora_linear(xd, wd, bank, idd), *plain(x, w, a, b, ids, ranks, scales), "with w")
    y0 = normal(gen, (T, N), dtype)
    y = y0.to(dtype).cuda()
    out = exm.lora_linear(xd, None, bank, idd, y=y)
    assert out is y
    ref, bound = plain(x, None, a, b, ids, ranks, scales, y0=y0)
    close(y, ref, bound, "added to y")
    none = (ids < 0) | (ranks[ids.clamp(min=0)] == 0)
    assert torch.equal(y.cpu()[none].double(), y0[none]), "a token without an adapter changed"


# (T, N, K): blocks of 16, 32 and 64, 128 x 128 and 256 x 256 tiles, all ragged
FORMS = [(70, 200, 136), (150, 700, 136), (150, 2604, 136), (601, 3804, 72), (4100, 4004, 64)]


@gpu
@pytest.mark.parametrize("order", ["one", "runs", "mixed", "distinct"])
@pytest.mark.parametrize("rank", [5, 16, 72, 128])
@pytest.mark.parametrize("T,N,K", FORMS)
def test_every_form(T, N, K, rank, order):
    """Token orders and ranks on every form, operands inside wider tensors of NaN."""
    print(f"lora forms T={T} N={N} K={K} rank={rank} order={order}", flush=True)
    gen = torch.Generator().manual_seed(rank)
    L, R = 24, (rank + 7) // 8 * 8
    x, w = whole(gen, (T, K), -1, 2), whole(gen, (N, K), -1, 2)
    a, b = whole(gen, (L, R, K), -1, 2), whole(gen, (L, N, R), -1, 2)
    ids = {"one": torch.full((T,), 3), "runs": torch.arange(T) // 21 % (L + 2) - 1,
           "mixed": torch.randint(-1, 4, (T,), generator=gen), "distinct": torch.arange(T) % L}[order]
    ranks = torch.full((L,), rank)
    ranks[1::5] = torch.tensor([0, 1, R, min(R, 17), 3])
    an, bn = a.clone(), b.clone()
    for i in range(L):
        an[i, ranks[i]:], bn[i, :, ranks[i]:] = float("nan"), float("nan")
    xw = torch.full((T, K + 24), float("nan"), dtype=BF16, device="cuda")
    xd = xw[:, 8:8 + K]
    xd.copy_(x)
    ww = torch.full((N, K + 8), float("nan"), dtype=BF16, device="cuda")
    ww[:, :K].copy_(w)
    bank = exm.LoraBank(an.to(BF16).cuda(), bn.to(BF16).cuda(), ranks=ranks.to(torch.int32).cuda())
    idd = ids.to(torch.int32).cuda()
    base, add = x @ w.t(), torch.zeros((T, N), dtype=torch.float64)
    for i in range(L):
        rows = ids == i
        if bool(rows.any()) and int(ranks[i]):
            r = int(ranks[i])
            add[rows] = (x[rows] @ a[i, :r].t()) @ b[i, :, :r].t()
    for pad in (8, 3):
        yw = torch.full((T + 2, N + pad), 9.0, dtype=BF16, device="cuda")
        y = yw[1:T + 1, pad // 2:pad // 2 + N]
        exm.lora_linear(xd, ww[:, :K], bank, idd, y=y)
        assert torch.equal(y.cpu(), (base + add).to(BF16)), "with w"
        y.copy_(base)
        y0 = y.cpu().double()
        exm.lora_linear(xd, None, bank, idd, y=y)
        assert torch.equal(y.cpu(), (y0 + add).to(BF16)), "added to y"
        y.fill_(9.0)
        assert bool((yw == 9).all()), "wrote outside its rows or columns"


@gpu
@pytest.mark.parametrize("T,N,K", [(150, 2604, 520), (601, 3804, 136), (1030, 2064, 1000)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_long_batches_against_fp64(T, N, K, dtype):
    print(f"lora long T={T} N={N} K={K} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(T)
    L, R = 7, 40
    x, w = normal(gen, (T, K), dtype), normal(gen, (N, K), dtype, 0.1)
    a, b = normal(gen, (L, R, K), dtype, 0.1), normal(gen, (L, N, R), dtype, 0.1)
    ranks, scales = torch.tensor([40, 0, 8, 33, 16, 24, 7]), torch.rand(L, generator=gen) * 3 - 1
    ids = torch.randint(-1, L, (T,), generator=gen)
    y = exm.lora_linear(x.to(dtype).cuda(), w.to(dtype).cuda(), device_bank(a, b, ranks, scales, dtype), ids.to(torch.int32).cuda())
    close(y, *plain(x, w, a, b, ids, ranks, scales.float().double()), "with w")


@gpu
@pytest.mark.parametrize("T,R", [(1, 8), (16, 128), (17, 24), (300, 40), (700, 128)])
def test_workspaces_are_enough(T, R):
    """A workspace of exactly the bytes asked for: what lies behind it stays as it was."""
    gen = torch.Generator().manual_seed(T)
    N, K, L = 3804, 72, 7
    x, w = whole(gen, (T, K), -1, 2), whole(gen, (N, K), -1, 2)
    a, b = whole(gen, (L, R, K), -1, 2), whole(gen, (L, N, R), -1, 2)
    ids = torch.randint(-1, L, (T,), generator=gen)
    need = exm.lora_workspace_bytes(T, N, K, L, R)
    buf = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    y = exm.lora_linear(x.to(BF16).cuda(), w.to(BF16).cuda(), exm.LoraBank(a.to(BF16).cuda(), b.to(BF16).cuda()),
                        ids.to(torch.int32).cuda(), workspace=buf[:need])
    ref, _ = plain(x, w, a, b, ids, torch.full((L,), R), torch.ones(L))
    assert torch.equal(y.cpu(), ref.to(BF16))
    assert bool((buf[need:] == 0xAB).all())


@gpu
def test_rows_far_apart():
    """Row strides of 2^24 elements, where no 32-bit offset spans the tokens."""
    gen = torch.Generator().manual_seed(3)
    T, N, K, L, R, ld = 101, 4 * 1664, 64, 3, 16, 1 << 24
    x, w = whole(gen, (T, K), -1, 2), whole(gen, (N, K), -1, 2)
    a, b = whole(gen, (L, R, K), -1, 2), whole(gen, (L, N, R), -1, 2)
    ids = torch.arange(T) % (L + 1) - 1
    xd = torch.empty((T - 1) * ld + K, dtype=BF16, device="cuda").as_strided((T, K), (ld, 1))
    xd.copy_(x)
    ref, _ = plain(x, w, a, b, ids, torch.full((L,), R), torch.ones(L))
    last = torch.empty(1 << 28, dtype=BF16, device="cuda").as_strided((1, K), (1 << 27, 1))   # one token: its stride means nothing
    last.copy_(x[:1])
    bank = exm.LoraBank(a.to(BF16).cuda(), b.to(BF16).cuda())
    assert torch.equal(exm.lora_linear(last, w.to(BF16).cuda(), bank, ids[:1].to(torch.int32).cuda()).cpu(), ref[:1].to(BF16))
    for n in (N, 1000):       # 64 x 64 and 16 x 16 blocks
        bank = exm.LoraBank(a.to(BF16).cuda(), b[:, :n].contiguous().to(BF16).cuda())
        y = exm.lora_linear(xd, w[:n].to(BF16).cuda(), bank, ids.to(torch.int32).cuda())
        assert torch.equal(y.cpu(), ref[:, :n].to(BF16))


@gpu
@pytest.mark.parametrize("order", ["one", "runs", "mixed", "distinct"])
@pytest.mark.parametrize("rank", [1, 7, 8, 9, 16, 31, 64, 128])
def test_whole_numbers_exact(order, rank):
    """Token orders: one adapter, runs of them that end inside a tile, mixed, all distinct."""
    print(f"lora whole numbers order={order} rank={rank}", flush=True)
    gen = torch.Generator().manual_seed(rank)
    T, N, K, L, R = 150, 96, 72, 160, (rank + 7) // 8 * 8
    x, w = whole(gen, (T, K), -1, 2), whole(gen, (N, K), -1, 2)
    a, b = whole(gen, (L, R, K), -1, 2), whole(gen, (L, N, R), -1, 2)
    a[:, rank:] = float("nan")           # what lies past the rank is not used
    b[:, :, rank:] = float("nan")
    ids = {"one": torch.full((T,), 3), "runs": torch.arange(T) // 21, "mixed": torch.randint(-1, 4, (T,), generator=gen),
           "distinct": torch.arange(T)}[order]
    ranks, scales = torch.full((L,), rank), torch.full((L,), 2.0)
    bank = device_bank(a, b, ranks, scales, FP16)
    y = exm.lora_linear(x.half().cuda(), w.half().cuda(), bank, ids.to(torch.int32).cuda())
    # |v| <= 72 and |sums| stay whole and small: hi + lo hold v exactly, so the only rounding
    # is the output's, and it is the same one on both sides
    ref, _ = plain(x, w, torch.nan_to_num(a), torch.nan_to_num(b), ids, ranks, scales)
    assert torch.equal(y.cpu(), ref.half())


@gpu
def test_other_tokens_and_adapters_do_not_leak():
    """NaN and infinities in one token, in adapters of other tokens and in unused ones."""
    gen = torch.Generator().manual_seed(2)
    T, N, K, L, R = 40, 80, 96, 6, 16
    x, w = whole(gen, (T, K)), whole(gen, (N, K))
    a, b = whole(gen, (L, R, K), -1, 2), whole(gen, (L, N, R), -1, 2)
    ids = torch.arange(T) % 4
    ids[7] = -1
    ids[9], ids[12] = L, -2147483648          # outside [0, L): no adapter
    ranks, scales = torch.full((L,), R), torch.ones(L)
    xd, wd = x.to(BF16).cuda(), w.to(BF16).cuda()
    ref, _ = plain(x, w, a, b, ids, ranks, scales)
    ad, bd = a.clone(), b.clone()
    ad[2], bd[3], ad[4], bd[5] = float("nan"), float("inf"), float("nan"), float("nan")
    xd[20] = float("nan")
    y = exm.lora_linear(xd, wd, device_bank(ad, bd, ranks, scales, BF16), ids.to(torch.int32).cuda()).cpu()
    keep = [t for t in range(T) if int(ids[t]) not in (2, 3) and t != 20]
    assert torch.equal(y[keep], ref[keep].to(BF16))
    assert bool(y[20].isnan().all())
    # an infinite v: the product is infinite or NaN, as the formula's is, in that token alone
    a2 = a.clone()
    x2 = x.clone()
    x2[5] = 0
    x2[5, 0] = 3e38
    a2[1, :, 0] = 3e38
    y = exm.lora_linear(x2.to(BF16).cuda(), wd, device_bank(a2, b, ranks, scales, BF16), ids.to(torch.int32).cuda()).cpu()
    keep = [t for t in range(T) if int(ids[t]) != 1]
    assert torch.equal(y[keep], ref[keep].to(BF16))


@gpu
def test_large_and_small_low_rank_values_in_fp16():
    """v beyond fp16's range, and far below it, with b that brings the result back."""
    gen = torch.Generator().manual_seed(5)
    T, N, K, L, R = 20, 48, 64, 2, 16
    x = normal(gen, (T, K), FP16, 8.0)
    w = normal(gen, (N, K), FP16, 0.1)
    a = torch.stack([normal(gen, (R, K), FP16, 8000.0), normal(gen, (R, K), FP16, 1e-6)])
    b = torch.stack([normal(gen, (N, R), FP16, 1e-5), normal(gen, (N, R), FP16, 30000.0)])
    ids, ranks, scales = torch.arange(T) % 2, torch.full((L,), R), torch.ones(L)
    ids[3] = -1
    y = exm.lora_linear(x.half().cuda(), w.half().cuda(), device_bank(a, b, ranks, scales, FP16),
                        ids.to(torch.int32).cuda())
    close(y, *plain(x, w, a, b, ids, ranks, scales), "fp16 range")


@gpu
@pytest.mark.parametrize("T", [5, 200])
def test_strides_defaults_and_offsets_past_32_bits(T):
    gen = torch.Generator().manual_seed(T)
    N, K, L, R = 72, 64, 3, 8
    x, w = whole(gen, (T, K)), whole(gen, (N, K))
    a, b = whole(gen, (L, R, K), -1, 2), whole(gen, (L, N, R), -1, 2)
    ids = torch.arange(T) % L
    ranks, scales = torch.full((L,), R), torch.ones(L)
    nan = float("nan")
    xw = torch.full((T, K + 24), nan, dtype=BF16, device="cuda")
    xd = xw[:, 8:8 + K]
    xd.copy_(x)
    ww = torch.full((N, K + 8), nan, dtype=BF16, device="cuda")
    ww[:, :K].copy_(w)
    stride = (1 << 31) + 512                               # adapters 2^32 bytes apart
    abuf = torch.empty(2 * stride + R * (K + 8), dtype=BF16, device="cuda")
    ad = abuf.as_strided((L, R, K), (stride, K + 8, 1))
    ad.copy_(a)
    bbuf = torch.empty(2 * stride + N * (R + 8), dtype=BF16, device="cuda")
    bd = bbuf.as_strided((L, N, R), (stride, R + 8, 1))
    bd.copy_(b)
    yw = torch.full((T, N + 3), 9.0, dtype=BF16, device="cuda")
    bank = exm.LoraBank(ad, bd)
    exm.lora_linear(xd, ww[:, :K], bank, ids.to(torch.int32).cuda(), y=yw[:, 1:N + 1])
    ref, _ = plain(x, w, a, b, ids, ranks, scales)
    assert torch.equal(yw[:, 1:N + 1].cpu(), ref.to(BF16))
    assert bool((yw[:, 0] == 9).all()) and bool((yw[:, N + 1:] == 9).all())


@gpu
@pytest.mark.parametrize("T", [1, 33, 260])
def test_streams_graphs_and_repeats(T):
    gen = torch.Generator().manual_seed(T + 70)
    N, K, L, R = 264, 512, 9, 32
    x = torch.randn((T, K), generator=gen).to(BF16).cuda()
    w = torch.randn((N, K), generator=gen).to(BF16).cuda()
    bank = exm.LoraBank(torch.randn((L, R, K), generator=gen).to(BF16).cuda(),
                        torch.randn((L, N, R), generator=gen).to(BF16).cuda())
    ids = torch.randint(-1, L, (T,), generator=gen).to(torch.int32).cuda()
    run = lambda: exm.lora_linear(x, w, bank, ids)
    first = run().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for i in range(4):
        x.mul_(0.5 if i % 2 else 2.0)
        ids.add_(1).remainder_(L)                          # other adapters at every replay
        want = run().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, captured), f"replay {i}"


@gpu
@pytest.mark.parametrize("T", [3, 37])
def test_adapters_beside_the_expert_layer(T):
    """Requests' adapters added to the output of the packed expert layer: y_moe + B A x."""
    from synthetic import TINY
    from tests.helpers import Layer, to_dev_bf16
    lay = Layer(TINY, seed=0, oracle_experts=False)
    s = lay.shape
    x = to_dev_bf16(lay.syn.x(T))
    base = exm.moe_layer(x, lay.wr, lay.bank, s.I, s.k).y
    gen = torch.Generator().manual_seed(1)
    L, R = 4, 16
    a, b = normal(gen, (L, R, s.H), BF16, 0.05), normal(gen, (L, s.H, R), BF16, 0.05)
    ids, ranks, scales = torch.arange(T) % (L + 1) - 1, torch.tensor([16, 8, 3, 0]), torch.ones(L)
    y0 = base.cpu().double()
    y = exm.lora_linear(x, None, device_bank(a, b, ranks, scales, BF16), ids.to(torch.int32).cuda(), y=base)
    close(y, *plain(x.cpu().double(), None, a, b, ids, ranks, scales, y0=y0), "layer + adapters")


@gpu
@pytest.mark.parametrize("T", [6, 150])
def test_one_adapter_equals_its_grouped_products(T):
    """Each adapter's part as two grouped products over the tokens sorted by adapter."""
    gen = torch.Generator().manual_seed(T)
    N, K, L, R = 136, 128, 5, 16
    x = whole(gen, (T, K), -1, 2).to(BF16).cuda()
    a, b = whole(gen, (L, R, K), -1, 2).to(BF16).cuda(), whole(gen, (L, N, R), -1, 2).to(BF16).cuda()
    ids = torch.randint(0, L, (T, 1), generator=gen).to(torch.int32).cuda()
    off, sf, f2s = exm.group_tokens(ids, L)
    v = exm.grouped_mm(x, a, off, row_index=sf)
    d = exm.grouped_mm(v, b, off)[f2s.long()]
    y = exm.lora_linear(x, None, exm.LoraBank(a, b), ids.view(-1), y=torch.zeros((T, N), dtype=BF16, device="cuda"))
    assert torch.equal(y, d)                               # |v| <= 128: bf16 holds it exactly
