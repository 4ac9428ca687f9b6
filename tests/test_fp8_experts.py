"""The experts in 8 bits (rms_norm, quantize_fp8, swiglu_fp8, quantize_fp8_weights, grouped_mm_fp8)
against plain forms in 64 bits, and a run of them as an expert layer.

Tolerances. e4m3 has steps of 2^-3 of a value's power of two down to 2^-6, and of 2^-9 below: t is off
by at most max(2^-4 |t|, 2^-10) when rounded (half a step). The quotient before it is formed with two
roundings (1 / scale, then the product) of 2^-24 and a division of up to 2^-23: 2^-21 |t| more.
Values that an operator computes before they are quantised are off by a relative delta of their own,
given at each test. The product's tolerances stand at product_bound()."""
import ctypes

import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16, FP16, FP32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
DTYPES = [BF16, FP16, FP32]
gpu = pytest.mark.gpu
INV, UNS = exm.ERR_INVALID_ARGUMENT, exm.ERR_UNSUPPORTED
# addresses far apart from each other, never dereferenced
X, W, Y, Q, S, R, RO, OFF, RI, XS, WS = (i << 40 for i in range(1, 12))


def groups_of(v, rows=1):
    """[..., n, K] padded with zeros to blocks of rows x 128: [..., nb, rows, kb, 128]."""
    n, K = v.shape[-2:]
    p = torch.nn.functional.pad(v, (0, -K % 128, 0, -n % rows))
    return p.view(*v.shape[:-2], (n + -n % rows) // rows, rows, (K + -K % 128) // 128, 128)


def spread(scale, n, K, rows=1):
    """A scale in front of each value: [..., nb, kb] -> [..., n, K]."""
    return scale.repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(128, -1)[..., :K]


def check_quantised(v, q, scale, delta, rows=1, weight=None, label=""):
    """q, scale against the values v (64 bits), themselves known to a relative delta."""
    q, scale = q.detach().cpu().to(FP32).double(), scale.detach().cpu().double()
    want = (groups_of(v, rows).abs().amax((-3, -1)) / 448).clamp(min=2.0 ** -126)
    w = torch.ones_like(want) if weight is None else weight.double()[:, None].expand_as(want)
    assert scale.shape == want.shape
    off = (scale - want * w).abs()
    assert bool((off <= (delta + 2.0 ** -23) * want * w.abs()).all()), f"{label}: scales off by {float((off / want).max()):.2e}"
    t = v / spread(want, v.shape[-2], v.shape[-1], rows)
    bad = (q - t).abs() > torch.clamp(2.0 ** -4 * t.abs(), min=2.0 ** -10) + (2 * delta + 2.0 ** -21) * t.abs()
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} of {bad.numel()} values off, first {bad.nonzero()[:3].tolist()}"


def close(got, ref, delta, label=""):
    got64 = got.detach().cpu().double()
    bound = delta * ref.abs()
    if got.dtype != FP32:
        fi = torch.finfo(got.dtype)
        bound = bound + fi.eps / 2 * (ref.abs() + bound).clamp(min=fi.tiny)
    bad = ~((got64 - ref).abs() <= bound)
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:3].tolist()}"


def randn(gen, *shape, sigma=1.0):
    return torch.randn(shape, generator=gen) * sigma


def on_gpu(v, shift=0, more=0, fill=float("nan")):
    """v on the GPU, its first element `shift` elements into an allocation, rows `more` elements longer."""
    n, K = v.shape[-2:]
    ld = K + more
    lead = v.shape[0] if v.dim() == 3 else 1
    buf = torch.full((shift + lead * n * ld,), fill, dtype=FP32, device="cuda").to(v.dtype)
    out = buf[shift:].view(*(() if v.dim() == 2 else (lead,)), n, ld)[..., :K]
    out.copy_(v)
    return out


# ------------------------------------------------------------------ refusals (no GPU)
def norm(x=X, ldx=256, w=W, wd=0, r=None, ldr=256, rd=0, ro=None, ldro=256, eps=1e-6, T=4, H=256, dt=0, y=Y, ldy=256, q=None,
         ldq=256, s=None, lds=2):
    return exm._lib.exmoe_rms_norm(exm._NORM.pack(*(v or 0 for v in (x, ldx, w, r, ldr, ro, ldro, y, ldy, q, ldq, s, lds)), eps, T, H,
                                                  dt, wd, rd), None)


def rows_of(x, ldx, w, ri, q, ldq, s, lds, n, rows, K, dt):
    return exm._FP8_ROWS.pack(*(v or 0 for v in (x, ldx, w, ri, q, ldq, s, lds)), n, rows, K, dt)


def quant(x=X, ldx=256, w=None, n=0, ri=None, rows=4, K=256, dt=0, q=Q, ldq=256, s=S, lds=2):
    return exm._lib.exmoe_quantize_fp8(rows_of(x, ldx, w, ri, q, ldq, s, lds, n, rows, K, dt), None)


def swiglu(x=X, ldx=512, w=None, n=0, ri=None, rows=4, I=256, dt=0, q=Q, ldq=256, s=S, lds=2):
    return exm._lib.exmoe_swiglu_fp8(rows_of(x, ldx, w, ri, q, ldq, s, lds, n, rows, I, dt), None)


def quantw(w=W, ldw=256, wst=256 * 100, E=3, N=100, K=256, dt=0, q=Q, ldq=256, qst=256 * 100, s=S, lds=2, sst=2):
    return exm._lib.exmoe_quantize_fp8_weights(
        exm._FP8_MATRICES.pack(*(v or 0 for v in (w, ldw, wst, q, ldq, qst, s, lds, sst)), E, N, K, dt), None)


def mm(x=X, ldx=256, xs=XS, ldxs=2, x_rows=8, ri=None, div=1, off=OFF, w=W, ldw=256, wst=256 * 100, ws=WS, ldws=2, wsst=2, rows=8,
       N=100, K=256, E=3, od=0, y=Y, ldy=100):
    return exm._lib.exmoe_grouped_mm_fp8(exm._GROUPED_FP8.pack(
        *(v or 0 for v in (x, ldx, xs, ldxs, ri, off, w, ldw, wst, ws, ldws, wsst, y, ldy)), x_rows, div, rows, N, K, E, od), None)


def test_the_structs_are_those_of_the_header():
    """Sizes of the C structs: pointers and sizes of 8 bytes, then 4-byte values, padded to 8."""
    for st, wide, narrow in ((exm._NORM, 13, 6), (exm._FP8_ROWS, 8, 4), (exm._FP8_MATRICES, 9, 4), (exm._GROUPED_FP8, 14, 7), (exm._BALANCE, 9, 5)):
        assert st.size == (8 * wide + 4 * narrow + 7) // 8 * 8
    for name in ("rms_norm", "quantize_fp8", "swiglu_fp8", "quantize_fp8_weights", "grouped_mm_fp8", "balance_loss_backward"):
        assert getattr(exm._lib, "exmoe_" + name)(None, None) == INV
    assert exm._lib.exmoe_balance_loss(None, None, 0, None) == INV


def refuses(call, status, **cases):
    for name, values in cases.items():
        for v in values:
            got = call(**(v if isinstance(v, dict) else {name: v}))
            assert got == status, (name, v, got, exm.last_error())


def test_refusals_of_the_norm():
    refuses(norm, INV, T=[-1], H=[0, -5], dt=[3, -1], wd=[1, 5], x=[None, X + 1], w=[None, W + 1], y=[Y + 1], ldx=[255], ldy=[100],
            eps=[-1.0, float("nan"), float("inf")], pair=[dict(q=Q), dict(s=S), dict(r=R), dict(ro=RO), dict(y=None)],
            fp8=[dict(q=Q, s=S, ldq=255), dict(q=Q, s=S + 2), dict(q=Q, s=S, lds=1)],
            res=[dict(r=R, ro=RO, rd=1), dict(r=R + 1, ro=RO), dict(r=R, ro=RO, ldr=200), dict(r=R, ro=RO, ldro=255)])
    refuses(norm, UNS, H=[16385], T=[1 << 22])
    assert norm(T=0, x=None, y=Y) == 0


def test_refusals_of_the_quantisers():
    refuses(quant, INV, rows=[-1], K=[0], dt=[3], x=[None, X + 1], q=[None], s=[None, S + 2], ldx=[255], ldq=[255], lds=[1])
    refuses(quant, UNS, K=[(1 << 24) + 1], big=[dict(rows=1 << 29)])
    refuses(swiglu, INV, rows=[-1], I=[0], dt=[7], ldx=[511], x=[None], lds=[1], w=[dict(w=W, n=3), dict(w=W + 2, n=4),
            dict(w=W, n=0, ri=RI), dict(ri=RI), dict(w=W, n=4, ri=RI + 1)])
    refuses(quantw, INV, E=[0], N=[0], K=[0], dt=[3], w=[None, W + 1], ldw=[255], wst=[100], qst=[100], sst=[1], lds=[1], q=[None],
            s=[None, S + 1])
    refuses(quantw, UNS, E=[65536], N=[(1 << 23) + 1])
    assert quant(rows=0, x=None) == 0 and swiglu(rows=0, x=None) == 0


def test_refusals_of_the_product():
    refuses(mm, INV, rows=[-1], N=[0], K=[0, 8, 100], E=[0, 257], od=[3], div=[0], x=[None, X + 8], w=[None, W + 8], xs=[None, XS + 2],
            ws=[None, WS + 1], ldx=[255, 264], ldw=[128, 260], wst=[100, 256 * 100 + 8], ldxs=[1], ldws=[1], wsst=[1], off=[None, OFF + 2],
            y=[None, Y + 1], ldy=[99], x_rows=[7], ri=[dict(ri=RI, x_rows=0), dict(ri=RI + 1)])
    refuses(mm, UNS, N=[(1 << 24) + 1], ldx=[(1 << 22) + 16], ldxs=[(1 << 20) + 1], ldws=[dict(ldws=(1 << 20) + 1, wsst=1 << 22)],
            tiles=[dict(rows=1 << 30, x_rows=1 << 30, N=1 << 24, ldy=1 << 24, wst=1 << 34, wsst=1 << 20),
                          # (fits as tiles, not as the smaller blocks that few rows per expert run on)
                          dict(rows=2560, x_rows=2560, N=6 << 20, K=16, ldx=16, ldw=16, ldxs=1, ldws=1, E=256, ldy=6 << 20,
                               wst=96 << 20, wsst=48 << 10)])
    assert mm(rows=0, x=None) == 0


def test_operands_that_share_memory_are_refused():
    def refused(status, *names):
        assert status == INV and exm.last_error() == "%s overlaps %s" % names, exm.last_error()

    refused(norm(y=X), "y", "x")
    refused(norm(r=R, ro=R + 2), "residual_out", "residual")
    refused(norm(r=R, ro=R, ldro=260), "residual_out", "residual")
    refused(norm(r=R, ro=X), "residual_out", "x")
    refused(norm(r=R, ro=W - 2 * 3 * 256 - 8), "residual_out", "w")
    refused(norm(q=Y + 4, s=S), "q", "y")
    refused(norm(q=Q, s=Q + 256 * 4 - 4), "scale", "q")
    refused(norm(q=Q, s=X), "scale", "x")
    refused(quant(q=X), "q", "x")
    refused(quant(s=Q), "q", "scale")
    refused(swiglu(w=S, n=4), "scale", "weights")
    refused(swiglu(w=W, n=40, ri=Q + 4), "q", "row_index")
    refused(quantw(q=W + 8), "q", "w")
    refused(quantw(s=W), "scale", "w")
    for at, name in ((X, "x"), (W, "w"), (XS, "x_scale"), (WS + 4, "w_scale"), (OFF, "expert_offsets")):
        refused(mm(y=at), "y", name)
    refused(mm(ri=Y + 4), "y", "row_index")


def test_a_tensor_that_asks_for_a_gradient_is_refused():
    x, w, v = torch.ones((4, 256), dtype=BF16), torch.ones(256, dtype=BF16), torch.ones(4)
    every = [((x, w), lambda: exm.rms_norm(x, w)), ((x,), lambda: exm.rms_norm(w, w, residual=x)), ((x,), lambda: exm.quantize_fp8(x)),
             ((x, v), lambda: exm.swiglu_fp8(x, v)), ((x,), lambda: exm.quantize_fp8_weights(x)),
             ((v,), lambda: exm.grouped_mm_fp8(x, v, x, v))]
    for tensors, call in every:
        for t in tensors:
            t.requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call()
            t.requires_grad_(False)


def test_8_bit_operands_that_ask_for_a_gradient_are_refused():
    x8, v = torch.ones((4, 256)).to(F8), torch.ones((4, 2))
    w8, ws = x8.view(1, 4, 256), v[:1].view(1, 1, 2)
    for t in (x8, w8):
        t.requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            exm.grouped_mm_fp8(x8.detach() if t is w8 else x8, v, w8.detach() if t is x8 else w8, ws)
        t.requires_grad_(False)
    with pytest.raises(ValueError, match="gradient"):
        exm.quantize_fp8_weights(torch.ones((1, 4, 256)), scale=torch.ones((1, 1, 2), requires_grad=True))


@gpu
def test_scales_that_ask_for_a_gradient_are_refused():
    x, w = torch.ones((4, 256), dtype=BF16, device="cuda"), torch.ones(256, dtype=BF16, device="cuda")
    for cols, call in ((2, lambda s: exm.quantize_fp8(x, scale=s)), (1, lambda s: exm.swiglu_fp8(x, scale=s)),
                       (2, lambda s: exm.rms_norm(x, w, out="fp8", scale=s))):
        s = torch.ones((4, cols), device="cuda", requires_grad=True)
        with pytest.raises(ValueError, match="gradient"):
            call(s)
        assert bool((s == 1).all())


@gpu
def test_refusals_of_the_binding():
    x, w = torch.ones((4, 256), dtype=BF16, device="cuda"), torch.ones(256, dtype=BF16, device="cuda")
    x8, xs = exm.quantize_fp8(x)
    w8, ws = exm.quantize_fp8_weights(x.view(1, 4, 256))
    bad = [lambda: exm.rms_norm(x, w[:128]), lambda: exm.rms_norm(x.t(), w), lambda: exm.rms_norm(x, w, out="fp4"),
           lambda: exm.rms_norm(x, w, residual=x[:2]), lambda: exm.rms_norm(x, w, residual_out=x), lambda: exm.rms_norm(x, w, q=x8),
           lambda: exm.rms_norm(x, w, out="fp8", y=x), lambda: exm.rms_norm(x.cpu(), w), lambda: exm.rms_norm(x, w, y=x.float()),
           lambda: exm.quantize_fp8(x, q=x8[:2]), lambda: exm.quantize_fp8(x, q=x), lambda: exm.quantize_fp8(x, scale=xs[:, :1]),
           lambda: exm.quantize_fp8(x.int()), lambda: exm.swiglu_fp8(x[:, :255]), lambda: exm.swiglu_fp8(x, weights=w),
           lambda: exm.swiglu_fp8(x, weights=xs, row_index=torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: exm.quantize_fp8_weights(x), lambda: exm.grouped_mm_fp8(x, xs, w8, ws), lambda: exm.grouped_mm_fp8(x8, xs[:2], w8, ws),
           lambda: exm.grouped_mm_fp8(x8, xs, w8, ws[:, :, :1]), lambda: exm.grouped_mm_fp8(x8[:, :128], xs, w8, ws),
           lambda: exm.grouped_mm_fp8(x8, xs, w8, ws, offsets=torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: exm.grouped_mm_fp8(x8, xs, w8, ws, out_dtype=F8), lambda: exm.grouped_mm_fp8(x8, xs, w8, ws, y=x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError, match="multiple of 16"):
        exm.grouped_mm_fp8(x8[:, :24], xs[:, :1], w8[..., :24], ws[..., :1])
    with pytest.raises(RuntimeError, match="aligned"):
        exm.grouped_mm_fp8(x8[:, 8:136], xs[:, :1], w8[..., :128], ws[..., :1])


# ------------------------------------------------------------------ quantisers
SIZES = [1, 7, 8, 100, 127, 128, 129, 1003, 2048]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 5, 67])
def test_rows_in_8_bits(rows, dtype):
    gen = torch.Generator().manual_seed(rows)
    for K in SIZES:
        for shift, more in ((0, 0), (1, 3)):
            x = randn(gen, rows, K, sigma=3.0).to(dtype)
            q, scale = exm.quantize_fp8(on_gpu(x, shift, more))
            check_quantised(x.double(), q, scale, 0.0, label=f"{rows} x {K}")
            assert q.stride(0) % 16 == 0 or rows == 1


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_values_at_the_borders(dtype):
    """Zeros, one value, the smallest and the largest ones, NaN and infinities, each group by itself."""
    fi = torch.finfo(dtype)
    x = torch.zeros((8, 384), dtype=dtype)
    x[0, 130] = 448.0
    x[0, 131:135] = torch.tensor([1.0, -17.0, 464.0 / 2, -26.0]).to(dtype)
    x[1, 5], x[1, 200] = fi.max, -fi.max
    x[2, :128], x[2, 128:256] = fi.tiny, fi.tiny / 4
    x[3, 3], x[3, 140] = float("nan"), 1.0
    x[4, 3], x[4, 4] = float("inf"), 1.0
    x[4, 300] = float("-inf")
    x[5] = torch.linspace(-448, 448, 384).to(dtype)
    x[6, 383] = -0.0
    q, scale = exm.quantize_fp8(x.cuda())
    fine = [0, 1, 2, 5, 6, 7]
    check_quantised(x[fine].double(), q[fine], scale[fine], 0.0)
    q, scale = q.float().cpu(), scale.cpu()
    assert bool((scale[7] == 2.0 ** -126).all()) and bool((q[7] == 0).all()) and bool((scale[0, 0::2] == 2.0 ** -126).all())
    assert scale[0, 1] == 1.0 and q[0, 130] == 448 and q[0, 131] == 1 and q[0, 132] in (-16, -18)
    assert torch.isnan(scale[3, 0]) and bool(torch.isnan(q[3, :128]).all()) and scale[3, 1] == torch.tensor(1.0) / 448
    assert q[3, 140] == 448 and not bool(torch.isnan(q[3, 128:]).any())
    assert torch.isinf(scale[4, 0]) and torch.isnan(q[4, 3]) and q[4, 4] == 0 and torch.isinf(scale[4, 2])
    assert bool(torch.isnan((q[4, :128].double() * scale[4, 0].double())).all()) and scale[4, 1] == 2.0 ** -126


@gpu
def test_only_the_outputs_are_written():
    gen = torch.Generator().manual_seed(3)
    for K in (24, 131, 256):
        x = randn(gen, 9, K).to(BF16).cuda()
        q = torch.full((11, K + 9), 7.0, device="cuda").to(F8)
        scale = torch.full((11, 5), -3.0, device="cuda")
        kb = (K + 127) // 128
        exm.quantize_fp8(x, q=q[1:10, 3:3 + K], scale=scale[1:10, 1:1 + kb])
        check_quantised(x.cpu().double(), q[1:10, 3:3 + K], scale[1:10, 1:1 + kb], 0.0)
        q, scale = q.float(), scale
        q[1:10, 3:3 + K], scale[1:10, 1:1 + kb] = 7.0, -3.0
        assert bool((q == 7).all()) and bool((scale == -3).all())


def swiglu_delta(g):
    """silu(g) u: 2^x of an argument rounded at |1.45 g| 2^-24 and off by 2^-23 itself, a reciprocal
    off by 2^-23, and four roundings."""
    return float((1.45 * g.abs().max() + 12) * 2.0 ** -24)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,I", [(1, 1), (1, 1024), (3, 127), (130, 200), (33, 1003), (257, 256)])
def test_gate_and_up_in_8_bits(rows, I, dtype):
    gen = torch.Generator().manual_seed(rows + I)
    x = randn(gen, rows, 2 * I, sigma=2.0).to(dtype)
    g, u = x.double().split(I, 1)
    h = g / (1 + torch.exp(-g)) * u
    for shift, more in ((0, 0), (1, 5)):
        xd = on_gpu(x, shift, more)
        q, scale = exm.swiglu_fp8(xd)
        check_quantised(h, q, scale, swiglu_delta(g), label="plain")
        weights = torch.rand((rows + 3) * 2, generator=gen)
        index = torch.randint(0, len(weights), (rows,), generator=gen).to(torch.int32)
        index[rows // 2] = -1 if rows % 2 else len(weights)        # no weight: zeros
        w = torch.where((index >= 0) & (index < len(weights)), weights[index.clamp(0, len(weights) - 1).long()], torch.tensor(0.0))
        q2, scale2 = exm.swiglu_fp8(xd, weights.cuda(), index.cuda())
        assert torch.equal(q2.float(), q.float())
        check_quantised(h, q2, scale2, swiglu_delta(g) + 2.0 ** -24, weight=w, label="indexed")
        q3, scale3 = exm.swiglu_fp8(xd, weights.cuda())
        check_quantised(h, q3, scale3, swiglu_delta(g) + 2.0 ** -24, weight=weights[:rows], label="in order")


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 128), (3, 100, 300), (2, 257, 129), (5, 384, 1008)])
def test_weights_in_8_bits(E, N, K, dtype):
    gen = torch.Generator().manual_seed(E + N + K)
    w = (randn(gen, E, N, K, sigma=0.02) * torch.exp(randn(gen, E, N, 1))).to(dtype)
    for shift, more in ((0, 0), (3, 1)):
        q, scale = exm.quantize_fp8_weights(on_gpu(w, shift, more))
        check_quantised(w.double(), q, scale, 0.0, rows=128)


# ------------------------------------------------------------------ norm
def norm_ref(x, w, eps, residual=None):
    h = x.double()
    if residual is not None:
        h = (x.float() + residual.float()).to(residual.dtype).double()
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()


# the sum of squares: 2 chunks of 8 one after another, then the lanes (8 steps) and at most 16 waves: under
# 50 roundings of 2^-24, half of them after the square root; division, root and products 6
NORM_DELTA = 31 * 2.0 ** -24


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 100, 512, 520, 1003, 1024, 2047, 2048, 2056, 4096, 6000, 8200, 16384])
def test_norm(H, dtype):
    gen = torch.Generator().manual_seed(H)
    for T, shift, more in ((1, 0, 0), (2, 1, 1), (9, 0, 8)):
        x = randn(gen, T, H, sigma=2.0).to(dtype)
        for wt in {dtype, FP32}:
            w = (1 + randn(gen, H, sigma=0.2)).to(wt)
            for rt in {None, dtype, FP32}:
                res = None if rt is None else randn(gen, T, H, sigma=3.0).to(rt)
                h, ref = norm_ref(x, w, 1e-5, res)
                label = f"{T} x {H} {dtype} {wt} {rt}"
                resd = None if res is None else on_gpu(res, shift, more)
                o = exm.rms_norm(on_gpu(x, shift, more), w.cuda(), 1e-5, residual=resd, out="both")
                close(o.y, ref, NORM_DELTA, label)
                check_quantised(ref, o.q, o.scale, NORM_DELTA, label=label)
                if rt is None:
                    assert o.residual is None
                    continue
                assert o.residual.dtype is rt and torch.equal(o.residual.cpu().double(), h), label
                assert torch.equal(resd.cpu(), res)
                again = exm.rms_norm(on_gpu(x), w.cuda(), 1e-5, residual=resd, out="y", residual_out=resd)      # in place
                assert again.residual is resd and torch.equal(resd.cpu().double(), h) and torch.equal(again.y, o.y)
                assert again.q is None and again.scale is None


@gpu
def test_norm_into_given_outputs():
    gen = torch.Generator().manual_seed(8)
    T, H = 7, 1000
    x, w = randn(gen, T, H).to(BF16), (1 + randn(gen, H, sigma=0.1)).to(BF16)
    _, ref = norm_ref(x, w, 1e-6)
    y = torch.full((T + 2, H + 3), 9.0, dtype=BF16, device="cuda")
    q, scale = torch.full((T + 2, H + 16), 7.0, device="cuda").to(F8), torch.full((T + 2, 10), -3.0, device="cuda")
    o = exm.rms_norm(x.cuda(), w.cuda(), out="both", y=y[1:-1, 1:H + 1], q=q[1:-1, 5:H + 5], scale=scale[1:-1, 1:9])
    close(y[1:-1, 1:H + 1], ref, NORM_DELTA)
    check_quantised(ref, q[1:-1, 5:H + 5], scale[1:-1, 1:9], NORM_DELTA)
    only = exm.rms_norm(x.cuda(), w.cuda(), out="fp8")
    assert torch.equal(only.q.float(), o.q.float()) and torch.equal(only.scale, o.scale) and only.y is None
    q = q.float()
    y[1:-1, 1:H + 1], q[1:-1, 5:H + 5], scale[1:-1, 1:9] = 9.0, 7.0, -3.0
    assert bool((y == 9).all()) and bool((q == 7).all()) and bool((scale == -3).all())


@gpu
def test_norm_of_special_rows():
    """A row of zeros, of one value, with a NaN, with an infinity: each row by itself."""
    H = 640
    x = torch.zeros((5, H), dtype=FP32)
    x[1, 77] = 3.0
    x[2], x[2, 9] = 1.0, float("nan")
    x[3], x[3, 200] = 1.0, float("inf")
    x[4] = 1e-30
    o = exm.rms_norm(x.cuda(), torch.ones(H, device="cuda"), out="both", eps=1e-6)
    y, q, s = o.y.cpu(), o.q.float().cpu(), o.scale.cpu()
    assert bool((y[0] == 0).all()) and bool((q[0] == 0).all()) and bool((s[0] == 2.0 ** -126).all())
    _, ref = norm_ref(x[1:2], torch.ones(H), 1e-6)
    close(y[1:2], ref, NORM_DELTA)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(s[2]).all()) and bool(torch.isnan(q[2]).all())
    assert torch.isnan(y[3, 200]) and bool((y[3, :200] == 0).all()) and torch.isnan(s[3, 1]) and not bool(torch.isnan(s[3, 2:]).any())
    _, ref = norm_ref(x[4:], torch.ones(H), 1e-6)
    close(y[4:], ref, NORM_DELTA)


# ------------------------------------------------------------------ product
def product_ref(x, xs, w, ws, offsets, src, cuts=False):
    """y and the products' magnitudes, in 64 bits; x, w the e4m3 values, src: the row of x of each row, -1: zeros."""
    rows, (E, N, K) = len(src), w.shape
    xv = x.double() * spread(xs.double(), x.shape[0], K)
    wv = w.double() * spread(ws.double(), N, K, 128)
    xr = torch.where((src >= 0)[:, None], xv[src.clamp(min=0)], torch.tensor(0.0, dtype=torch.float64))
    y, mag, cut = (torch.zeros((rows, N), dtype=torch.float64) for _ in range(3))
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            y[a:b] = xr[a:b] @ wv[e].t()
            if cuts:
                mag[a:b] = xr[a:b].abs() @ wv[e].abs().t()
            for k in range(0, K if cuts else 0, 8):     # the largest product of each 8 neighbours
                part = xr[a:b, None, k:k + 8].abs() * wv[e][None, :, k:k + 8].abs()
                cut[a:b] += part.amax(-1)
    return y, mag, cut


def product_bound(y, mag, cut, K, dtype):
    """fp32 sums: K + 2 roundings of 2^-23 of what is summed (as in the 16-bit products) and three of
    the scales. 16-bit outputs: the matrix unit cuts each of 8 neighbouring products at 2^-13 of the
    largest of them, 2^-10 of the largest in all; and half a step of the result."""
    bound = mag * (K + 5) * 2.0 ** -23
    if dtype != FP32:
        fi = torch.finfo(dtype)
        bound = bound + cut * 2.0 ** -10
        bound = bound + fi.eps / 2 * (y.abs() + bound).clamp(min=fi.tiny)
    return bound


def f8(v):
    return v.to(F8)


def offsets_of(counts):
    return torch.tensor([0] + counts).cumsum(0).to(torch.int32)


def check_product(x, xs, w, ws, counts, dtype, row_index=None, row_div=1, exact=False, ragged=0, label=""):
    off = offsets_of(counts)
    rows = int(off[-1]) if row_index is None else len(row_index)
    src = torch.arange(rows) if row_index is None else torch.where(row_index >= 0, row_index // row_div, -1).long()
    src = torch.where(src < x.shape[0], src, -1)
    y, mag, cut = product_ref(x.float(), xs, w.float(), ws, off, src, cuts=not exact)
    yd = torch.full((rows, w.shape[1] + ragged), 7.0, dtype=dtype, device="cuda")[:, ragged // 2:w.shape[1] + ragged // 2]
    ri = None if row_index is None else row_index.cuda()
    xd, wd = (on_gpu(t, 0, 16 * bool(ragged)) for t in (x, w))
    exm.grouped_mm_fp8(xd, on_gpu(xs, 0, ragged), wd, on_gpu(ws, 0, ragged), off.cuda(), row_index=ri, row_div=row_div, y=yd, out_dtype=dtype)
    got = yd.cpu().double()
    if exact:
        assert torch.equal(got, y.to(dtype).double()), f"{label}: {int((got != y.to(dtype).double()).sum())} of {y.numel()} differ"
    else:
        bad = ~((got - y).abs() <= product_bound(y, mag, cut, w.shape[2], dtype))
        assert not bool(bad.any()), f"{label}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:4].tolist()}"


def whole_operands(gen, rows, E, N, K):
    """Small whole numbers and scales of powers of two: sums are exact."""
    kb, nb = (K + 127) // 128, (N + 127) // 128
    x = f8(torch.randint(-2, 3, (rows, K), generator=gen).float())
    w = f8(torch.randint(-2, 3, (E, N, K), generator=gen).float())
    xs = 2.0 ** torch.randint(-2, 3, (rows, kb), generator=gen).float()
    ws = 2.0 ** torch.randint(-2, 3, (E, nb, kb), generator=gen).float()
    return x, xs, w, ws


PRODUCTS = [([1], 1, 16), ([1], 16, 16), ([1], 128, 128), ([3, 0, 1], 40, 272), ([0, 0, 0, 2], 517, 128), ([16], 256, 2048),
            ([17, 1, 40, 0, 9], 200, 400), ([130], 130, 144), ([200, 3, 64], 384, 640), ([300], 64, 1008), ([515, 257], 256, 256),
            ([1] * 60 + [0] * 4, 48, 256), ([2500], 136, 128), ([40] * 30, 640, 144), ([90, 0, 130, 77] * 4, 4100, 128),
            ([1200, 3, 900], 6700, 160), ([2049], 6400, 272), ([5, 0, 3], 200, 2064), ([9, 2, 12, 1], 3100, 4112), ([100, 2, 30], 264, 2320)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,N,K", PRODUCTS)
def test_product_of_whole_numbers(counts, N, K, dtype):
    gen = torch.Generator().manual_seed(N + K)
    x, xs, w, ws = whole_operands(gen, sum(counts), len(counts), N, K)
    check_product(x, xs, w, ws, counts, dtype, exact=True, label="plain")
    check_product(x, xs, w, ws, counts, dtype, exact=True, ragged=3, label="ragged rows")
    k = 3
    T = sum(counts) + 5
    x, xs, _, _ = whole_operands(gen, T, 1, 1, K)
    index = torch.randint(0, T * k, (sum(counts),), generator=gen).to(torch.int32)
    index[0] = -1
    index[-1] = T * k + 7
    check_product(x, xs, w, ws, counts, dtype, row_index=index, row_div=k, exact=True, label="gathered")


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,N,K", [([1], 64, 256), ([5, 0, 20], 130, 400), ([90], 256, 1024), ([300, 40], 136, 272)])
def test_product_of_normal_values(counts, N, K, dtype):
    gen = torch.Generator().manual_seed(N * K)
    x, xs = randn(gen, sum(counts), K), None
    w = randn(gen, len(counts), N, K, sigma=0.02)
    x8, xs = exm.quantize_fp8(x.cuda())
    w8, ws = exm.quantize_fp8_weights(w.cuda())
    check_product(x8.cpu(), xs.cpu(), w8.cpu(), ws.cpu(), counts, dtype)


@gpu
def test_one_matrix_without_offsets():
    gen = torch.Generator().manual_seed(2)
    for rows, N, K in ((1, 256, 512), (33, 100, 144), (400, 384, 256)):
        x, xs, w, ws = whole_operands(gen, rows, 1, N, K)
        y, _, _ = product_ref(x.float(), xs, w.float(), ws, offsets_of([rows]), torch.arange(rows))
        got = exm.grouped_mm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda())
        assert got.dtype is BF16 and torch.equal(got.cpu().double(), y.to(BF16).double())


@gpu
def test_rows_outside_the_segments_are_left():
    gen = torch.Generator().manual_seed(5)
    rows, N, K = 300, 130, 256
    x, xs, w, ws = whole_operands(gen, rows, 3, N, K)
    for off in ([0, 20, 20, 200], [10, 20, 120, 290], [0, 0, 0, 0], [300, 300, 300, 300]):
        offsets = torch.tensor(off, dtype=torch.int32)
        y, _, _ = product_ref(x.float(), xs, w.float(), ws, offsets, torch.arange(rows))
        y = y.to(BF16)
        y[:off[0]], y[off[3]:] = 5.0, 5.0
        got = exm.grouped_mm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), offsets.cuda(), y=torch.full((rows, N), 5.0, dtype=BF16, device="cuda"))
        assert torch.equal(got.cpu(), y), off
    for off in ([-5, 100, 400, 1000], [0, 250, 100, 300]):       # no grouping: nothing leads out of the buffers
        exm.grouped_mm_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), torch.tensor(off, dtype=torch.int32).cuda())


@gpu
@pytest.mark.parametrize("rows", [3, 200])
def test_a_nan_stays_in_its_row_and_column(rows):
    gen = torch.Generator().manual_seed(rows)
    N, K = 192, 384
    x, xs, w, ws = whole_operands(gen, rows, 1, N, K)
    y, _, _ = product_ref(x.float(), xs, w.float(), ws, offsets_of([rows]), torch.arange(rows))
    for dtype in (BF16, FP32):
        xf, wf, xs2, ws2 = x.float(), w.float(), xs.clone(), ws.clone()
        xf[1, 200], wf[0, 40, 3] = float("nan"), float("nan")
        xs2[2, 1] = float("inf")
        ws2[0, 1, 2] = float("nan")                              # columns 128 and up
        got = exm.grouped_mm_fp8(f8(xf).cuda(), xs2.cuda(), f8(wf).cuda(), ws2.cuda(), out_dtype=dtype).cpu()
        fine = torch.ones((rows, N), dtype=torch.bool)
        fine[1], fine[2], fine[:, 40], fine[:, 128:] = False, False, False, False
        assert torch.equal(got[fine], y.to(dtype)[fine])
        assert bool(torch.isnan(got[1]).all()) and bool(torch.isnan(got[:, 40]).all()) and bool(torch.isnan(got[:, 128:]).all())
        assert not bool(torch.isfinite(got[2]).any())


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_of_x_beyond_32_bit_offsets(dtype):
    """x of 2.2 GiB behind row_index: rows at its start, around 2 GiB and at its end; zeros elsewhere."""
    gen = torch.Generator().manual_seed(13)
    N, K, rows = 200, 2048, 1150000
    at = torch.tensor([0, 3, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, rows - 2, rows - 1])
    x, xs, w, ws = whole_operands(gen, len(at), 2, N, K)
    xd = torch.zeros((rows, K), dtype=torch.uint8, device="cuda").view(F8)
    sd = torch.zeros((rows, K // 128), device="cuda")
    xd.view(torch.uint8)[at.cuda()] = x.view(torch.uint8).cuda()
    sd[at.cuda()] = xs.cuda()
    pick = torch.randint(0, len(at), (150,), generator=gen)
    index = at[pick].to(torch.int32)
    index[7], index[8], index[9] = -1, rows, 77
    src = torch.where(torch.arange(150) == 9, len(at), torch.where((index < 0) | (index >= rows), -1, pick))
    off = offsets_of([60, 90])
    y, _, _ = product_ref(torch.cat([x.float(), torch.zeros((1, K))]), torch.cat([xs, torch.zeros((1, K // 128))]), w.float(), ws, off, src)
    got = exm.grouped_mm_fp8(xd, sd, w.cuda(), ws.cuda(), off.cuda(), row_index=index.cuda(), out_dtype=dtype)
    assert torch.equal(got.cpu().double(), y.to(dtype).double())


@gpu
def test_equal_calls_give_equal_bits():
    gen = torch.Generator().manual_seed(9)
    x8, xs = exm.quantize_fp8(randn(gen, 500, 1024).cuda())
    w8, ws = exm.quantize_fp8_weights(randn(gen, 4, 512, 1024).cuda())
    off = offsets_of([100, 0, 399, 1]).cuda()
    first = exm.grouped_mm_fp8(x8, xs, w8, ws, off, out_dtype=FP32)
    for _ in range(3):
        assert torch.equal(exm.grouped_mm_fp8(x8, xs, w8, ws, off, out_dtype=FP32), first)


# ------------------------------------------------------------------ together
def expert_layer(exm, x, res, wn, wr, gu8, gus, d8, ds, k, E):
    """A layer of experts in 8 bits behind its norm, as a user joins the calls."""
    n = exm.rms_norm(x, wn, residual=res, out="both")
    _, ids, weights = exm.route_topk(n.y, wr, k)
    offsets, sorted_flat, flat_to_sorted = exm.group_tokens(ids, E)
    gate_up = exm.grouped_mm_fp8(n.q, n.scale, gu8, gus, offsets, row_index=sorted_flat, row_div=k)
    h, hs = exm.swiglu_fp8(gate_up, weights, sorted_flat)
    rows = exm.grouped_mm_fp8(h, hs, d8, ds, offsets, out_dtype=FP32)
    y = rows[flat_to_sorted.long()].view(x.shape[0], k, -1).sum(1)
    return y, n, ids, weights


def layer_operands(gen, T, H, I, E):
    x, res = randn(gen, T, H).to(BF16).cuda(), randn(gen, T, H, sigma=2.0).to(BF16).cuda()
    wn, wr = (1 + randn(gen, H, sigma=0.1)).to(BF16).cuda(), randn(gen, E, H, sigma=0.05).to(BF16).cuda()
    gu, d = randn(gen, E, 2 * I, H, sigma=0.05).cuda(), randn(gen, E, H, I, sigma=0.05).cuda()
    return x, res, wn, wr, *exm.quantize_fp8_weights(gu), *exm.quantize_fp8_weights(d)


@gpu
@pytest.mark.parametrize("T", [1, 16, 200])
def test_an_expert_layer(T):
    """The norm against 64 bits, and the layer against 64 bits without any quantisation of the
    activations. A rounding to e4m3 is off by 2^-3 / sqrt(12) of the value's power of two, 2.7% of values
    spread over it: that of x reaches gate and up, sqrt(2) 2.7%, that of their product 2.7%; together
    4.7% of the result's norm."""
    H, I, E, k = 256, 256, 8, 2
    gen = torch.Generator().manual_seed(T)
    x, res, wn, wr, gu8, gus, d8, ds = layer_operands(gen, T, H, I, E)
    y, n, ids, weights = expert_layer(exm, x, res, wn, wr, gu8, gus, d8, ds, k, E)
    h, ref = norm_ref(x.cpu(), wn.cpu(), 1e-6, res.cpu())
    close(n.y, ref, NORM_DELTA)
    assert torch.equal(n.residual.cpu().double(), h)
    gu = gu8.cpu().float().double() * spread(gus.cpu().double(), 2 * I, H, 128)
    d = d8.cpu().float().double() * spread(ds.cpu().double(), H, I, 128)
    want = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            g, u = (gu[e] @ ref[t]).split(I)
            want[t] += float(weights[t, j]) * (d[e] @ (g / (1 + torch.exp(-g)) * u))
    off = float((y.cpu().double() - want).norm() / want.norm())
    assert off < 0.06, off


@gpu
def test_an_expert_layer_captured_and_on_another_stream():
    T, H, I, E, k = 24, 256, 128, 8, 2
    gen = torch.Generator().manual_seed(1)
    args = layer_operands(gen, T, H, I, E)
    eager = [t.clone() for t in (lambda r: (r[0], r[1].y, r[1].scale, r[1].residual))(expert_layer(exm, *args, k, E))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = expert_layer(exm, *args, k, E)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], eager[0]) and torch.equal(got[1].y, eager[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, n, _, _ = expert_layer(exm, *args, k, E)
    for i in range(4):
        args[0].copy_(randn(gen, T, H).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        again = expert_layer(exm, *args, k, E)
        assert torch.equal(y, again[0]) and torch.equal(n.y, again[1].y) and torch.equal(n.scale, again[1].scale)
        assert torch.equal(n.residual, again[1].residual) and torch.equal(n.q.float(), again[1].q.float())
