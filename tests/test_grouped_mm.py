"""Products grouped by expert and their gradients (grouped_mm, grouped_mm_dgrad,
grouped_mm_wgrad) against a plain fp64 loop over the experts.

Tolerances. Inputs are 16-bit values, so products are exact in fp32; a sum of R of them in
fp32 is off by at most R roundings of partial sums, each at most 2^-24 S with
S = sum |a||b| when rounded to nearest and 2^-23 S when an adder drops the bits below: R 2^-23
S. A 16-bit output adds half a step, eps / 2 of its value (taken of |ref| + the first term);
below the smallest normal number the step no longer shrinks with the value: it stays at
eps x tiny (fp16: 2^-10 2^-14 = 2^-24), so half of it, eps / 2 x tiny, is the least half step.
Small whole numbers are summed without any rounding: those results are equal bit for bit."""
import ctypes

import numpy as np
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

FAKE = 0x10000   # aligned, never dereferenced: validation fails before any enqueue
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
gpu = pytest.mark.gpu


# ------------------------------------------------------------------ plain forms (fp64, CPU)
def segments(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def plain_mm(x, w, offsets, src):
    rows = len(src)
    y = torch.zeros((rows, w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e, a, b in segments(offsets):
        y[a:b] = x[src[a:b]] @ w[e].t()
        mag[a:b] = x[src[a:b]].abs() @ w[e].abs().t()
    return y, mag * w.shape[2] * 2.0 ** -23


def plain_dgrad(dy, w, offsets, f2s=None, k=1):
    dx = torch.zeros((dy.shape[0], w.shape[2]), dtype=torch.float64)
    mag = torch.zeros_like(dx)
    for e, a, b in segments(offsets):
        dx[a:b] = dy[a:b] @ w[e]
        mag[a:b] = dy[a:b].abs() @ w[e].abs()
    n = w.shape[1]
    if f2s is not None:
        dx, mag = dx[f2s.long()].view(-1, k, w.shape[2]).sum(1), mag[f2s.long()].view(-1, k, w.shape[2]).sum(1)
        n += k
    return dx, mag * n * 2.0 ** -23


def plain_wgrad(dy, x, offsets, src):
    E = len(offsets) - 1
    dw = torch.zeros((E, dy.shape[1], x.shape[1]), dtype=torch.float64)
    bound = torch.zeros_like(dw)
    for e, a, b in segments(offsets):
        dw[e] = dy[a:b].t() @ x[src[a:b]]
        bound[e] = (dy[a:b].abs().t() @ x[src[a:b]].abs()) * (b - a + 16) * 2.0 ** -23
    return dw, bound


def close(got, ref, bound, label):
    got64 = got.detach().cpu().double()
    assert got64.shape == ref.shape, (label, got64.shape, ref.shape)
    if got.dtype != FP32:
        fi = torch.finfo(got.dtype)
        bound = bound + fi.eps / 2 * (ref.abs() + bound).clamp(min=fi.tiny)
    bad = ~((got64 - ref).abs() <= bound)
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} outside the bound, first {bad.nonzero()[:4].tolist()}"


def equal(got, ref, label):
    want = ref.to(got.dtype)
    g = got.detach().cpu()
    assert torch.equal(g, want), f"{label}: {int((g != want).sum())} of {g.numel()} differ, first {(g != want).nonzero()[:4].tolist()}"


def whole(gen, shape, lo=-2, hi=3):
    return torch.randint(lo, hi, shape, generator=gen).double()


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def routed(gen, T, k, E):
    """ids, offsets, sorted_flat, flat_to_sorted of a random routing, by plain sorting."""
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)])
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    f2s = torch.empty_like(order)
    f2s[order] = torch.arange(T * k)
    offs = offsets_of(torch.bincount(flat, minlength=E).tolist())
    return ids.to(torch.int32), offs, order.to(torch.int32), f2s.to(torch.int32)


# ------------------------------------------------------------------ refusals (no GPU)
def _mm(x=FAKE, ldx=64, x_rows=8, ri=None, div=1, off=FAKE, w=FAKE, ldw=64, ws=64 * 32, rows=8, N=32, K=64, E=2, dt=0,
        out=0, y=FAKE, ldy=32):
    return exm._lib.exmoe_grouped_mm(x, ldx, x_rows, ri, div, off, w, ldw, ws, rows, N, K, E, dt, out, y, ldy, None, 0,
                                     None)


def _dg(dy=FAKE, lddy=32, off=FAKE, w=FAKE, ldw=64, ws=64 * 32, f2s=None, k=1, rows=8, N=32, K=64, E=2, dt=0, out=0,
        dx=FAKE, lddx=64, wsp=None, wsb=0):
    return exm._lib.exmoe_grouped_mm_dgrad(dy, lddy, off, w, ldw, ws, f2s, k, rows, N, K, E, dt, out, dx, lddx, wsp, wsb,
                                           None)


def _wg(dy=FAKE, lddy=32, x=FAKE, ldx=64, x_rows=8, ri=None, div=1, off=FAKE, rows=8, N=32, K=64, E=2, dt=0, out=2,
        dw=FAKE, lddw=64, dws=64 * 32, wsp=None, wsb=0):
    return exm._lib.exmoe_grouped_mm_wgrad(dy, lddy, x, ldx, x_rows, ri, div, off, rows, N, K, E, dt, out, dw, lddw, dws,
                                           wsp, wsb, None)


@pytest.mark.parametrize("call", [_mm, _dg, _wg])
def test_shared_refusals(call):
    inv = exm.ERR_INVALID_ARGUMENT
    for bad in (dict(rows=-1), dict(N=0), dict(K=-3), dict(E=0), dict(E=257), dict(dt=2), dict(dt=5), dict(out=1),
                dict(out=7), dict(off=None), dict(off=FAKE + 2)):
        assert call(**bad) == inv, bad
        assert exm.last_error() != ""
    assert call(N=(1 << 24) + 1) == exm.ERR_UNSUPPORTED


def test_mm_refusals():
    inv = exm.ERR_INVALID_ARGUMENT
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x=FAKE + 1), dict(y=FAKE + 1), dict(y=FAKE + 2, out=2),
                dict(ldx=63), dict(ldw=63), dict(ldy=31), dict(ws=64 * 32 - 1), dict(div=0), dict(x_rows=7),
                dict(ri=FAKE, x_rows=0), dict(ri=FAKE + 1)):
        assert _mm(**bad) == inv, bad
    assert _mm(rows=0) == exm.OK
    assert _mm(rows=0, x=None, y=None, off=None) == exm.OK
    # more output tiles than a launch holds: refused before anything runs
    assert _mm(rows=1 << 30, x_rows=1 << 30, N=1 << 24, ldy=1 << 24, ws=1 << 40) == exm.ERR_UNSUPPORTED


def test_dgrad_refusals():
    inv = exm.ERR_INVALID_ARGUMENT
    for bad in (dict(dy=None), dict(w=None), dict(dx=None), dict(lddy=31), dict(lddx=63), dict(f2s=FAKE, k=3),
                dict(f2s=FAKE, k=0), dict(f2s=FAKE + 2, k=2)):
        assert _dg(**bad) == inv, bad
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_DGRAD, 8, 32, 64, 2, 2)
    assert need > 0
    assert _dg(f2s=FAKE, k=2) == exm.ERR_WORKSPACE and str(need) in exm.last_error()
    assert _dg(f2s=FAKE, k=2, wsp=FAKE, wsb=need - 1) == exm.ERR_WORKSPACE
    assert _dg(f2s=FAKE, k=2, wsp=FAKE + 4, wsb=need) == inv
    assert _dg(rows=0) == exm.OK


def test_wgrad_refusals():
    inv = exm.ERR_INVALID_ARGUMENT
    for bad in (dict(dy=None), dict(x=None), dict(dw=None), dict(lddy=31), dict(ldx=63), dict(lddw=63),
                dict(dws=64 * 32 - 1), dict(x_rows=7), dict(div=0), dict(dw=FAKE + 2)):
        assert _wg(**bad) == inv, bad
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_WGRAD, 1 << 16, 32, 64, 2, 0)
    assert need > 0, "few tiles over many rows split the sum"
    assert _wg(rows=1 << 16, x_rows=1 << 16) == exm.ERR_WORKSPACE


def test_odd_row_lengths_need_a_workspace():
    """Operands whose rows are no multiple of 8 elements are copied with padded rows first."""
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_MM, 512, 32, 63, 2)
    assert need >= (512 * 64 + 2 * 32 * 64) * 2
    assert _mm(rows=512, x_rows=512, K=63) == exm.ERR_WORKSPACE and str(need) in exm.last_error()
    for op, call in ((exm.GROUPED_DGRAD, _dg), (exm.GROUPED_WGRAD, _wg)):
        for n, k in ((31, 64), (32, 63), (31, 63)):
            need = exm.grouped_mm_workspace_bytes(op, 8, n, k, 2, 0)
            assert need > 0
            assert call(N=n, K=k) == exm.ERR_WORKSPACE and str(need) in exm.last_error()


def test_workspace_query_of_bad_arguments():
    assert exm.grouped_mm_workspace_bytes(3, 8, 8, 8, 2) == 0
    assert exm.grouped_mm_workspace_bytes(exm.GROUPED_DGRAD, 8, 8, 8, 300, 1) == 0
    assert exm.grouped_mm_workspace_bytes(exm.GROUPED_MM, 8, 8, 8, 2) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    x, w = torch.zeros(4, 8, dtype=BF16), torch.zeros(2, 16, 8, dtype=BF16)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        exm.grouped_mm(x, w, off)
    with pytest.raises(ValueError, match="axes"):
        exm.grouped_mm(x[0], w, off)


# ------------------------------------------------------------------ GPU
def cuda(t, dtype):
    return t.to(dtype).cuda()


COUNTS = [[0, 1, 130, 0, 17, 64, 0], [1], [0, 0], [5, 260]]
SIZES = [(1, 1), (8, 64), (63, 65), (129, 200), (300, 515), (256, 128), (136, 72), (2, 1000)]


@gpu
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (FP16, FP16)])
def test_whole_numbers_exact(counts, N, K, dtype, out):
    print(f"whole numbers counts={counts} N={N} K={K} {dtype} -> {out}", flush=True)
    gen = torch.Generator().manual_seed(N * 1000 + K)
    E, rows = len(counts), sum(counts)
    off = offsets_of(counts)
    x, w, dy = whole(gen, (rows, K)), whole(gen, (E, N, K)), whole(gen, (rows, N))
    src = torch.arange(rows)
    xd, wd, dyd, offd = cuda(x, dtype), cuda(w, dtype), cuda(dy, dtype), off.cuda()
    equal(exm.grouped_mm(xd, wd, offd, out_dtype=out), plain_mm(x, w, off, src)[0], "mm")
    equal(exm.grouped_mm_dgrad(dyd, wd, offd, out_dtype=out), plain_dgrad(dy, w, off)[0], "dgrad")
    equal(exm.grouped_mm_wgrad(dyd, xd, offd, out_dtype=out), plain_wgrad(dy, x, off, src)[0], "wgrad")


@gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 8, 64), (65, 6, 13), (300, 8, 256), (700, 2, 3)])
@pytest.mark.parametrize("N,K", [(256, 192), (77, 131)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_routed_batch_against_fp64(T, k, E, N, K, dtype):
    print(f"routed T={T} k={k} E={E} N={N} K={K} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(T * 31 + N)
    ids, off, order, f2s = routed(gen, T, k, E)
    x = torch.randn((T, K), generator=gen).to(dtype).double()
    w = (torch.randn((E, N, K), generator=gen) * 0.05).to(dtype).double()
    dy = torch.randn((T * k, N), generator=gen).to(dtype).double()
    src = order.long() // k
    xd, wd, dyd = cuda(x, dtype), cuda(w, dtype), cuda(dy, dtype)
    o, sf, fs = exm.group_tokens(ids.cuda(), E)          # the library's own grouping feeds the products
    assert torch.equal(o.cpu(), off) and torch.equal(sf.cpu(), order) and torch.equal(fs.cpu(), f2s)
    for out in (dtype, FP32):
        close(exm.grouped_mm(xd, wd, o, row_index=sf, row_div=k, out_dtype=out), *plain_mm(x, w, off, src), f"mm {out}")
        close(exm.grouped_mm_dgrad(dyd, wd, o, out_dtype=out), *plain_dgrad(dy, w, off), f"dgrad rows {out}")
        close(exm.grouped_mm_dgrad(dyd, wd, o, flat_to_sorted=fs, k=k, out_dtype=out),
              *plain_dgrad(dy, w, off, f2s, k), f"dgrad tokens {out}")
        close(exm.grouped_mm_wgrad(dyd, xd, o, row_index=sf, row_div=k, out_dtype=out),
              *plain_wgrad(dy, x, off, src), f"wgrad {out}")


@gpu
@pytest.mark.parametrize("rows", [511, 4096, 20000])
def test_wgrad_long_sums(rows):
    """Few small experts over many rows: the sum is split and joined, equal bits every time."""
    gen = torch.Generator().manual_seed(rows)
    counts = [rows // 3, 0, rows - rows // 3 - 5, 5]
    off = offsets_of(counts)
    dy, x = torch.randn((rows, 40), generator=gen).to(BF16).double(), torch.randn((rows, 72), generator=gen).to(BF16).double()
    dyd, xd, offd = cuda(dy, BF16), cuda(x, BF16), off.cuda()
    got = exm.grouped_mm_wgrad(dyd, xd, offd)
    close(got, *plain_wgrad(dy, x, off, torch.arange(rows)), "wgrad")
    assert torch.equal(got, exm.grouped_mm_wgrad(dyd, xd, offd)), "not repeatable"
    close(exm.grouped_mm_wgrad(dyd, xd, offd, out_dtype=BF16), *plain_wgrad(dy, x, off, torch.arange(rows)), "wgrad bf16")


def strided(t, dtype, pad_front, pad_back, value=float("nan")):
    """t as the inside of a wider tensor whose other columns hold `value`."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad_front + pad_back,), value, dtype=dtype, device="cuda")
    view = wide[..., pad_front:pad_front + t.shape[-1]]
    view.copy_(t)
    return wide, view


@gpu
@pytest.mark.parametrize("front,back", [(0, 8), (8, 8), (1, 0), (3, 2), (0, 1)])
@pytest.mark.parametrize("N,K", [(64, 136), (30, 77)])
def test_strides_and_alignments(front, back, N, K):
    print(f"strides front={front} back={back} N={N} K={K}", flush=True)
    gen = torch.Generator().manual_seed(9)
    counts = [33, 0, 90]
    off, rows, E = offsets_of(counts), 123, 3
    x, w, dy = whole(gen, (rows, K)), whole(gen, (E, N, K)), whole(gen, (rows, N))
    src = torch.arange(rows)
    _, xd = strided(x, BF16, front, back)
    _, dyd = strided(dy, BF16, front, back)
    wide = torch.full((E, N + 3, K + front + back), float("nan"), dtype=BF16, device="cuda")
    wd = wide[:, 1:N + 1, front:front + K]
    wd.copy_(w)
    offd = off.cuda()
    for op, ref in (("mm", plain_mm(x, w, off, src)[0]), ("dgrad", plain_dgrad(dy, w, off)[0]),
                    ("wgrad", plain_wgrad(dy, x, off, src)[0])):
        for out in (FP32, BF16):
            ow, ov = strided(torch.zeros(ref.shape), out, front, back, 7.0)
            if op == "mm":
                exm.grouped_mm(xd, wd, offd, out_dtype=out, y=ov)
            elif op == "dgrad":
                exm.grouped_mm_dgrad(dyd, wd, offd, out_dtype=out, dx=ov)
            else:
                exm.grouped_mm_wgrad(dyd, xd, offd, out_dtype=out, dw=ov)
            equal(ov, ref, f"{op} {out}")
            edge = torch.cat([ow[..., :front].flatten(), ow[..., front + ref.shape[-1]:].flatten()])
            assert bool((edge == 7.0).all()), f"{op}: wrote outside its columns"


@gpu
@pytest.mark.parametrize("counts", [[300, 0, 210], [20, 3, 44]])
@pytest.mark.parametrize("front,back", [(1, 7), (3, 2)])
def test_misaligned_rows_of_whole_length(counts, front, back):
    """Row lengths that are multiples of 8 at addresses that are not, few and many rows."""
    print(f"misaligned counts={counts} front={front} back={back}", flush=True)
    gen = torch.Generator().manual_seed(14)
    E, rows, N, K = 3, sum(counts), 144, 136
    off, src = offsets_of(counts), torch.arange(sum(counts))
    x, w, dy = whole(gen, (rows, K)), whole(gen, (E, N, K)), whole(gen, (rows, N))
    xd, dyd, wd = (strided(t, FP16, front, back)[1] for t in (x, dy, w))
    offd = off.cuda()
    equal(exm.grouped_mm(xd, wd, offd, out_dtype=FP32), plain_mm(x, w, off, src)[0], "mm")
    equal(exm.grouped_mm_dgrad(dyd, wd, offd, out_dtype=FP32), plain_dgrad(dy, w, off)[0], "dgrad")
    equal(exm.grouped_mm_wgrad(dyd, xd, offd), plain_wgrad(dy, x, off, src)[0], "wgrad")


@gpu
def test_rows_outside_the_segments():
    """Offsets that start after row 0 and end before the last: those rows stay as they were,
    what they hold reaches no output, and experts without rows may hold anything."""
    gen = torch.Generator().manual_seed(3)
    N, K, rows = 72, 136, 300
    off = torch.tensor([10, 10, 90, 90, 201], dtype=torch.int32)
    x, w, dy = whole(gen, (rows, K)), whole(gen, (4, N, K)), whole(gen, (rows, N))
    src = torch.arange(rows)
    ref_y, ref_dx, ref_dw = plain_mm(x, w, off, src)[0], plain_dgrad(dy, w, off)[0], plain_wgrad(dy, x, off, src)[0]
    nan = float("nan")
    xd, wd, dyd, offd = cuda(x, BF16), cuda(w, BF16), cuda(dy, BF16), off.cuda()
    for t in (xd, dyd):
        t[:10] = nan
        t[201:] = nan
    wd[0] = nan
    wd[2] = nan
    y = torch.full((rows, N), 5.0, dtype=BF16, device="cuda")
    exm.grouped_mm(xd, wd, offd, y=y)
    equal(y[10:201], ref_y[10:201], "mm")
    assert bool((y[:10] == 5).all()) and bool((y[201:] == 5).all())
    dx = torch.full((rows, K), 5.0, dtype=BF16, device="cuda")
    exm.grouped_mm_dgrad(dyd, wd, offd, dx=dx)
    equal(dx[10:201], ref_dx[10:201], "dgrad")
    assert bool((dx[:10] == 5).all()) and bool((dx[201:] == 5).all())
    equal(exm.grouped_mm_wgrad(dyd, xd, offd), ref_dw, "wgrad")


@gpu
def test_broken_offsets_and_indices_stay_in_bounds():
    """Offsets past the rows, below zero or falling, and indices outside x: no access leaves
    the buffers; rows of a bad index are zeros and an ungrouped row adds nothing."""
    gen = torch.Generator().manual_seed(4)
    N, K, rows = 40, 48, 64
    x, w, dy = whole(gen, (8, K)), whole(gen, (3, N, K)), whole(gen, (rows, N))
    xd, wd, dyd = cuda(x, BF16), cuda(w, BF16), cuda(dy, BF16)
    bad = torch.tensor([-5, 30, 20, 1 << 30], dtype=torch.int32)
    idx = torch.randint(0, 8, (rows,), generator=gen).to(torch.int32)
    idx[[3, 40]] = torch.tensor([-1, 8], dtype=torch.int32)
    y = torch.full((rows, N), 5.0, dtype=FP32, device="cuda")
    exm.grouped_mm(xd, wd, bad.cuda(), row_index=idx.cuda(), out_dtype=FP32, y=y)
    use = [s for s in range(rows) if s not in (3, 40)]
    ref = torch.zeros((rows, N), dtype=torch.float64)
    for s in use:
        ref[s] = w[0 if s < 20 else 2] @ x[idx[s]]
    # rows 20..29 belong to expert 0's segment and expert 2's: either result is theirs
    both = [s for s in use if not 20 <= s < 30]
    equal(y[both], ref[both], "mm")
    assert bool((y[3] == 0).all()) and bool((y[40] == 0).all())
    off = torch.tensor([0, 20, 20, rows], dtype=torch.int32)
    dw = exm.grouped_mm_wgrad(dyd, xd, off.cuda(), row_index=idx.cuda())
    refw = torch.zeros((3, N, K), dtype=torch.float64)
    for s in use:
        refw[0 if s < 20 else 2] += torch.outer(dy[s], x[idx[s]])
    equal(dw, refw, "wgrad")
    f2s = torch.randperm(rows, generator=gen).to(torch.int32)
    f2s[[0, 7]] = torch.tensor([-1, rows], dtype=torch.int32)
    off2 = torch.tensor([0, 20, 20, rows - 4], dtype=torch.int32)      # the last four rows are ungrouped
    dx = exm.grouped_mm_dgrad(dyd, wd, off2.cuda(), flat_to_sorted=f2s.cuda(), k=4, out_dtype=FP32)
    rd = torch.zeros((rows // 4, K), dtype=torch.float64)
    for f in range(rows):
        s = int(f2s[f])
        if 0 <= s < rows - 4:
            rd[f // 4] += dy[s] @ w[0 if s < 20 else 2]
    equal(dx, rd, "dgrad")


@gpu
def test_infinities_stay_in_their_rows():
    gen = torch.Generator().manual_seed(6)
    counts, N, K = [70, 60], 64, 96
    off, rows = offsets_of(counts), 130
    x, w = whole(gen, (rows, K)), whole(gen, (2, N, K), 1, 3)
    xd, wd = cuda(x, BF16), cuda(w, BF16)
    xd[5, 3], xd[100, 90] = float("inf"), float("nan")
    y = exm.grouped_mm(xd, wd, off.cuda(), out_dtype=FP32)
    ref = plain_mm(x, w, off, torch.arange(rows))[0]
    keep = [s for s in range(rows) if s not in (5, 100)]
    equal(y[keep], ref[keep], "mm")
    assert bool((y[5] == float("inf")).all()) and bool(y[100].isnan().all())


@gpu
@pytest.mark.parametrize("dtype,unit", [(FP16, 2.0 ** -24), (BF16, 2.0 ** -133)])
def test_subnormal_inputs_count(dtype, unit):
    """Multiples of the smallest subnormal are not taken for zeros."""
    gen = torch.Generator().manual_seed(7)
    off, N, K = offsets_of([20, 30]), 48, 40
    x, w, dy = whole(gen, (50, K)), whole(gen, (2, N, K)), whole(gen, (50, N))
    big = 2.0 ** 10 if dtype is FP16 else 2.0 ** 100
    src = torch.arange(50)
    xd, wd, dyd = cuda(x * unit, dtype), cuda(w * big, dtype), cuda(dy * big, dtype)
    equal(exm.grouped_mm(xd, wd, off.cuda(), out_dtype=FP32), plain_mm(x * unit, w * big, off, src)[0], "mm")
    equal(exm.grouped_mm_wgrad(dyd, xd, off.cuda()), plain_wgrad(dy * big, x * unit, off, src)[0], "wgrad")


@gpu
def test_offsets_past_32_bits():
    """An expert stride and a row stride that lead past 2^32 bytes."""
    gen = torch.Generator().manual_seed(8)
    N, K, stride, ld = 24, 40, (1 << 31) + 64, (1 << 26) + 8
    off = offsets_of([3, 37])
    w, x, dy = whole(gen, (2, N, K)), whole(gen, (40, K)), whole(gen, (40, N))
    wbuf = torch.empty(stride + N * K, dtype=BF16, device="cuda")
    wd = wbuf.as_strided((2, N, K), (stride, K, 1))
    wd.copy_(w)
    xbuf = torch.empty(39 * ld + K, dtype=BF16, device="cuda")
    xd = xbuf.as_strided((40, K), (ld, 1))
    xd.copy_(x)
    dyd, src = cuda(dy, BF16), torch.arange(40)
    equal(exm.grouped_mm(xd, wd, off.cuda(), out_dtype=FP32), plain_mm(x, w, off, src)[0], "mm")
    equal(exm.grouped_mm_dgrad(dyd, wd, off.cuda(), out_dtype=FP32), plain_dgrad(dy, w, off)[0], "dgrad")
    equal(exm.grouped_mm_wgrad(dyd, xd, off.cuda()), plain_wgrad(dy, x, off, src)[0], "wgrad")
    ybuf = torch.empty(39 * ld + N, dtype=BF16, device="cuda")
    y = ybuf.as_strided((40, N), (ld, 1))
    exm.grouped_mm(xd, wd, off.cuda(), y=y)
    equal(y, plain_mm(x, w, off, src)[0], "mm into wide rows")


TALL = [250, 0, 1, 700, 321, 320, 319, 33, 640, 257, 256, 288, 32, 322, 99, 161]   # about 250 on average

# (counts, N, K): 16-row blocks and 64 x 64 blocks (few tiles), tiles of 128, 256 and 320 rows in
# each direction, split and whole sums over the rows; ragged edges everywhere; odd row lengths,
# few and many rows per expert.
FORMS = [([3, 0, 9, 1], 72, 136), ([100, 0, 37, 201], 200, 264),
         ([100, 0, 37, 201], 840, 264), ([100, 0, 37, 201], 264, 840), ([130, 0, 1000, 1, 600], 904, 136),
         ([130, 0, 1000, 1, 600], 136, 904), ([1, 4199], 4104, 72), ([4200], 72, 4104), ([0, 1600], 2824, 2824),
         (TALL, 4616, 72), (TALL, 72, 4616),
         ([200, 0, 190], 41, 77), ([200, 0, 190], 40, 77), ([30, 0, 90], 200, 77), ([9, 200, 2], 41, 80), ([700, 690], 523, 129), ([1, 2], 41, 77),
         ([0, 2500], 130, 1001)]


@gpu
@pytest.mark.parametrize("counts,N,K", FORMS)
@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (FP16, FP16)])
def test_every_form_with_a_gather_nan_neighbours_and_bad_indices(counts, N, K, dtype, out):
    """Operands inside wider tensors of NaN, rows before the first and behind the last segment,
    x gathered through an index with two entries outside it; outputs into wider tensors."""
    print(f"forms counts={counts} N={N} K={K} {dtype} -> {out}", flush=True)
    gen = torch.Generator().manual_seed(N * 7 + K)
    E, grouped = len(counts), sum(counts)
    lead, rows, xr = 4, grouped + 4 + 3, grouped // 2 + 1
    off = offsets_of(counts) + lead
    x, w, dy = whole(gen, (xr, K), -1, 2), whole(gen, (E, N, K), -1, 2), whole(gen, (rows, N), -1, 2)
    idx = torch.randint(0, 2 * xr, (rows,), generator=gen).to(torch.int32)
    src = idx.long() // 2
    bad = [lead, lead + grouped - 1] if grouped > 3 else []
    idx[bad] = torch.tensor([-1, 2 * xr], dtype=torch.int32)[:len(bad)]
    odd = 1 if K % 8 else 8
    xw, xd = strided(x, dtype, odd, 8)
    _, dyd = strided(dy, dtype, 1 if N % 8 else 8, 8)
    dyd[:lead], dyd[lead + grouped:] = float("nan"), float("nan")
    _, wd = strided(w, dtype, odd, 8)
    offd, idxd = off.cuda(), idx.cuda()
    xz = torch.cat([x, torch.zeros((1, K), dtype=torch.float64)])     # a bad index: zeros
    src[bad] = xr
    ref_y, ref_dx, ref_dw = plain_mm(xz, w, off, src)[0], plain_dgrad(dy, w, off)[0], plain_wgrad(dy, xz, off, src)[0]
    inner = slice(lead, lead + grouped)
    for pad in (8, 3):
        yw, y = strided(torch.zeros((rows, N)), out, pad, 8, 7.0)
        y.fill_(7.0)
        exm.grouped_mm(xd, wd, offd, row_index=idxd, row_div=2, out_dtype=out, y=y)
        equal(y[inner], ref_y[inner], "mm")
        y[inner] = 7.0
        assert bool((yw == 7).all()), "mm wrote outside its rows or columns"
        dxw, dx = strided(torch.zeros((rows, K)), out, pad, 8, 7.0)
        dx.fill_(7.0)
        exm.grouped_mm_dgrad(dyd, wd, offd, out_dtype=out, dx=dx)
        equal(dx[inner], ref_dx[inner], "dgrad")
        dx[inner] = 7.0
        assert bool((dxw == 7).all()), "dgrad wrote outside its rows or columns"
        dww, dw = strided(torch.zeros((E, N, K)), out, pad, 8, 7.0)
        exm.grouped_mm_wgrad(dyd, xd, offd, row_index=idxd, row_div=2, out_dtype=out, dw=dw)
        equal(dw, ref_dw, "wgrad")
        dw.fill_(7.0)
        assert bool((dww == 7).all()), "wgrad wrote outside its columns"


@gpu
@pytest.mark.parametrize("counts,N,K", [([100, 0, 37, 203], 200, 264), ([100, 0, 37, 203], 264, 840),
                                        ([130, 1, 1000, 601], 136, 904), ([200, 0, 192], 41, 77),
                                        ([2, 4198], 72, 4104)])
def test_token_gradients_of_every_form(counts, N, K):
    """The gradient of x summed per token (k = 4), with ungrouped rows and an index outside."""
    print(f"token gradients counts={counts} N={N} K={K}", flush=True)
    gen = torch.Generator().manual_seed(K)
    rows, E, k = sum(counts), len(counts), 4
    off = offsets_of(counts)
    off[-1] -= 1                                                       # the last row is ungrouped
    w, dy = whole(gen, (E, N, K), -1, 2), whole(gen, (rows, N), -1, 2)
    f2s = torch.randperm(rows, generator=gen).to(torch.int32)
    f2s[5] = rows
    dyd = cuda(dy, BF16)
    dyd[-1] = float("nan")
    got = exm.grouped_mm_dgrad(dyd, cuda(w, BF16), off.cuda(), flat_to_sorted=f2s.cuda(), k=k, out_dtype=FP32)
    per_row = torch.cat([plain_dgrad(dy, w, off)[0], torch.zeros((1, K), dtype=torch.float64)])
    equal(got, per_row[f2s.long()].view(-1, k, K).sum(1), "dgrad")


@gpu
def test_infinite_rows_far_apart():
    """Few summed rows 2^27 elements apart, the first of them infinite: positions past the last
    row are zeros times zeros, not zeros times the first row."""
    inf, ld = float("inf"), 1 << 27
    buf = torch.empty(7 * ld + 64, dtype=BF16, device="cuda")
    rows8 = buf.as_strided((8, 64), (ld, 1))
    rows8.fill_(1.0)
    rows8[0] = inf
    near = torch.ones((8, 64), dtype=BF16, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    dx = exm.grouped_mm_dgrad(near[:, :8], rows8.unsqueeze(0), off, out_dtype=FP32)
    assert bool((dx == inf).all())
    many = torch.ones((400, 8), dtype=BF16, device="cuda")
    dx = exm.grouped_mm_dgrad(many, rows8.unsqueeze(0), torch.tensor([0, 400], dtype=torch.int32, device="cuda"), out_dtype=FP32)
    assert bool((dx == inf).all())
    assert bool((exm.grouped_mm_wgrad(rows8, near, off) == inf).all())
    assert bool((exm.grouped_mm_wgrad(near, rows8, off) == inf).all())
    one = buf.as_strided((1, 64), (1 << 31, 1))       # one row: its stride means nothing
    off1 = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert bool((exm.grouped_mm_wgrad(one, near[:1], off1) == inf).all())
    assert bool((exm.grouped_mm_wgrad(near[:1], one, off1) == inf).all())


@gpu
def test_no_rows_and_no_routing():
    """No rows at all: nothing is written but the zeros of a gradient of W; a routing that gives
    every row to nobody does the same."""
    w, off = torch.ones((2, 40, 72), dtype=BF16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    none, some = torch.empty((0, 72), dtype=BF16, device="cuda"), torch.ones((50, 72), dtype=BF16, device="cuda")
    assert exm.grouped_mm(none, w, off).shape == (0, 40)
    assert exm.grouped_mm_dgrad(none[:, :40], w, off).shape == (0, 72)
    for x in (none, some):
        dy = torch.full((len(x), 40), float("nan"), dtype=BF16, device="cuda")
        dw = torch.full((2, 40, 72), 5.0, device="cuda")
        exm.grouped_mm_wgrad(dy, x, off, dw=dw)
        assert bool((dw == 0).all())
    y = torch.full((50, 40), 5.0, dtype=BF16, device="cuda")
    exm.grouped_mm(some, w, off, y=y)
    assert bool((y == 5).all())
    dx = exm.grouped_mm_dgrad(y, w, off, flat_to_sorted=torch.arange(50, dtype=torch.int32, device="cuda"), k=5)
    assert dx.shape == (10, 72) and bool((dx == 0).all())


@gpu
@pytest.mark.parametrize("N,K", [(131, 203), (64, 203), (131, 64), (64, 64)])
def test_workspaces_are_enough(N, K):
    """A workspace of exactly the bytes asked for: what lies behind it stays as it was."""
    gen = torch.Generator().manual_seed(15)
    counts, k = [700, 0, 1300], 4
    rows, E, off = sum(counts), len(counts), offsets_of(counts)
    x, w, dy = whole(gen, (rows, K)), whole(gen, (E, N, K)), whole(gen, (rows, N))
    xd, wd, dyd, offd, src = cuda(x, BF16), cuda(w, BF16), cuda(dy, BF16), off.cuda(), torch.arange(rows)
    f2s = torch.randperm(rows, generator=gen).to(torch.int32)

    def guarded(op, kk, run):
        need = exm.grouped_mm_workspace_bytes(op, rows, N, K, E, kk)
        buf = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
        out = run(buf[:need])
        assert bool((buf[need:] == 0xAB).all())
        return out

    equal(guarded(exm.GROUPED_MM, 0, lambda ws: exm.grouped_mm(xd, wd, offd, out_dtype=FP32, workspace=ws)),
          plain_mm(x, w, off, src)[0], "mm")
    equal(guarded(exm.GROUPED_DGRAD, 0, lambda ws: exm.grouped_mm_dgrad(dyd, wd, offd, out_dtype=FP32, workspace=ws)),
          plain_dgrad(dy, w, off)[0], "dgrad rows")
    equal(guarded(exm.GROUPED_DGRAD, k, lambda ws: exm.grouped_mm_dgrad(dyd, wd, offd, flat_to_sorted=f2s.cuda(), k=k,
                                                                        out_dtype=FP32, workspace=ws)),
          plain_dgrad(dy, w, off, f2s, k)[0], "dgrad tokens")
    equal(guarded(exm.GROUPED_WGRAD, 0, lambda ws: exm.grouped_mm_wgrad(dyd, xd, offd, workspace=ws)),
          plain_wgrad(dy, x, off, src)[0], "wgrad")


@gpu
def test_two_calls_at_once():
    """Two streams, each with outputs and a workspace of its own, at the same time."""
    gen = torch.Generator().manual_seed(12)
    T, k, E, N, K = 150, 4, 6, 131, 203
    ids, off, order, f2s = routed(gen, T, k, E)
    x, w, dy = torch.randn((T, K), generator=gen), torch.randn((E, N, K), generator=gen), torch.randn((T * k, N), generator=gen)
    xd, wd, dyd, offd, sf, fs = cuda(x, BF16), cuda(w, BF16), cuda(dy, BF16), off.cuda(), order.cuda(), f2s.cuda()
    need = max(exm.grouped_mm_workspace_bytes(op, T * k, N, K, E, k) for op in range(3))

    def run(scale, ws):
        return (exm.grouped_mm(xd * scale, wd, offd, row_index=sf, row_div=k, workspace=ws),
                exm.grouped_mm_dgrad(dyd * scale, wd, offd, flat_to_sorted=fs, k=k, workspace=ws),
                exm.grouped_mm_wgrad(dyd * scale, xd, offd, row_index=sf, row_div=k, workspace=ws))

    spaces = [exm.alloc_workspace(need) for _ in range(2)]
    want = [[t.clone() for t in run(s, spaces[0])] for s in (1.0, 2.0)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(float(i + 1), spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@gpu
@pytest.mark.parametrize("T,k,E,N,K", [(90, 4, 9, 136, 264), (150, 4, 3, 131, 203)])
def test_streams_graphs_and_repeats(T, k, E, N, K):
    """Equal bits on another stream and on every replay of a captured graph, also when the
    inputs change between replays and other work runs in between."""
    gen = torch.Generator().manual_seed(11)
    k = min(k, E)
    ids, off, order, f2s = routed(gen, T, k, E)
    dev = dict(x=torch.randn((T, K), generator=gen).to(BF16).cuda(), w=torch.randn((E, N, K), generator=gen).to(BF16).cuda(),
               dy=torch.randn((T * k, N), generator=gen).to(BF16).cuda())
    offd, sf, fs = off.cuda(), order.cuda(), f2s.cuda()
    ws = exm.alloc_workspace(exm.grouped_mm_workspace_bytes(exm.GROUPED_DGRAD, T * k, N, K, E, k))

    def run():
        return (exm.grouped_mm(dev["x"], dev["w"], offd, row_index=sf, row_div=k),
                exm.grouped_mm_dgrad(dev["dy"], dev["w"], offd, flat_to_sorted=fs, k=k, workspace=ws),
                exm.grouped_mm_wgrad(dev["dy"], dev["x"], offd, row_index=sf, row_div=k))

    first = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for i in range(4):
        dev["x"].mul_(0.5 if i % 2 else 2.0)
        want = [t.clone() for t in run()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured)), f"replay {i}"


@gpu
def test_expert_layer_step_forward_and_backward():
    """The products as a training step uses them on dense experts: route, group, gate and up,
    SwiGLU, down, routing weights, and the gradients of tokens and weights, against autograd
    in fp64 and against differences of the fp64 loss."""
    gen = torch.Generator().manual_seed(21)
    T, H, I, E, k = 24, 128, 64, 8, 2
    x = torch.randn((T, H), generator=gen).to(BF16)
    wr = (torch.randn((E, H), generator=gen) * 0.1).to(BF16)
    w1 = (torch.randn((E, 2 * I, H), generator=gen) * 0.1).to(BF16)
    w2 = (torch.randn((E, H, I), generator=gen) * 0.1).to(BF16)
    gy = torch.randn((T, H), generator=gen)
    _, ids, wts = exm.route_topk(x.cuda(), wr.cuda(), k)
    off, sf, fs = exm.group_tokens(ids, E)
    xd, w1d, w2d = x.cuda(), w1.cuda(), w2.cuda()
    gu = exm.grouped_mm(xd, w1d, off, row_index=sf, row_div=k, out_dtype=FP32)
    sg = torch.sigmoid(gu[:, :I])
    h = (gu[:, :I] * sg * gu[:, I:]).to(BF16)
    o = exm.grouped_mm(h, w2d, off, out_dtype=FP32)
    y = (o[fs.long()].view(T, k, H) * wts.unsqueeze(2)).sum(1)
    # backward: routed rows take their token's gradient times the routing weight
    tok = (sf // k).long()
    do = (gy.cuda()[tok] * wts.view(-1)[sf.long()].unsqueeze(1)).to(BF16)
    dh = exm.grouped_mm_dgrad(do, w2d, off, out_dtype=FP32)
    dw2 = exm.grouped_mm_wgrad(do, h, off)
    dgate = dh * gu[:, I:] * sg * (1 + gu[:, :I] * (1 - sg))
    dup = dh * gu[:, :I] * sg
    dgu = torch.cat([dgate, dup], 1).to(BF16)
    dx = exm.grouped_mm_dgrad(dgu, w1d, off, flat_to_sorted=fs, k=k, out_dtype=FP32)
    dw1 = exm.grouped_mm_wgrad(dgu, xd, off, row_index=sf, row_div=k)

    X, W1, W2 = (t.double().requires_grad_() for t in (x, w1, w2))
    idc, wc = ids.cpu().long(), wts.cpu().double()

    def loss(X, W1, W2):
        out = []
        for t in range(T):
            acc = 0
            for j in range(k):
                e = idc[t, j]
                g = W1[e] @ X[t]
                hh = torch.nn.functional.silu(g[:I]) * g[I:]
                acc = acc + wc[t, j] * (W2[e] @ hh)
            out.append(acc)
        out = torch.stack(out)
        return out, (out * gy.double()).sum()

    ref, value = loss(X, W1, W2)
    value.backward()

    # One 16-bit rounding of h, do or dgu is 2^-8 of each term of the sums behind it; two of
    # them meet in dw and dx (do, then dgu; or h and do), and a random sign on each term leaves
    # far less than the sum of absolute terms: 3 2^-8 of the largest magnitude covers both.
    def near(got, want, label):
        err = (got.detach().cpu().double() - want).abs().max() / want.abs().max()
        print(f"  {label}: {err:.2e}", flush=True)
        assert err <= 3 * 2.0 ** -8, label

    near(y, ref.detach(), "y")
    near(dx, X.grad, "dx")
    near(dw1, W1.grad, "dw1")
    near(dw2, W2.grad, "dw2")
    d = 1e-4
    for leaf, got in ((0, dx), (1, dw1), (2, dw2)):
        direction = torch.randn(got.shape, generator=gen).double()
        args = [X.detach(), W1.detach(), W2.detach()]
        up, dn = list(args), list(args)
        up[leaf], dn[leaf] = args[leaf] + d * direction, args[leaf] - d * direction
        diff = (loss(*up)[1] - loss(*dn)[1]) / (2 * d)
        along = (got.cpu().double() * direction).sum()
        # the direction sums got.numel() roundings of random sign: 4 standard deviations
        tol = 4 * 2.0 ** -8 * (got.cpu().double() * direction).norm()
        assert (diff - along).abs() <= tol, (leaf, float(diff), float(along), float(tol))
