"""The expert layer in 8 bits (moe_layer_fp8): bit for bit what its calls give one by one, in place, captured and
on another stream; near the layer in 64 bits without quantised activations; its refusals."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16, FP32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu
INV, UNS = exm.ERR_INVALID_ARGUMENT, exm.ERR_UNSUPPORTED
AT = {name: i << 40 for i, name in enumerate(("x", "w_norm", "residual", "w_router", "logit_bias", "gate_up", "gate_up_scale", "down",
                                              "down_scale", "logits", "topk_ids", "topk_weights", "expert_offsets", "sorted_flat",
                                              "flat_to_sorted", "y", "ws"), 1)}


def call(T=4, H=256, I=128, E=8, k=2, eps=1e-6, wsb=None, ws=AT["ws"], **at):
    p = {**{n: v for n, v in AT.items() if n != "ws"}, **at}
    need = exm._lib.exmoe_moe_layer_fp8_workspace_bytes(T, H, I, E, k)
    return exm._lib.exmoe_moe_layer_fp8(exm._LAYER_FP8.pack(*(v or 0 for v in p.values()), eps, T, H, I, E, k, 1), ws,
                                        need if wsb is None else wsb, None)


def test_refusals():
    assert exm._LAYER_FP8.size == 160 and exm._lib.exmoe_moe_layer_fp8(None, None, 0, None) == INV
    for bad in (dict(T=-1), dict(H=0), dict(H=200), dict(I=100), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**bad) == INV, bad
    for bad in (dict(H=16384 + 128), dict(I=32768), dict(T=1 << 22), dict(E=128, k=65), dict(T=1 << 21, k=8, E=8, I=16384)):
        assert call(**bad) == UNS, bad
    # (2^33 threads for the sums of the rows: more than one launch)
    assert call(T=(1 << 22) - 1, H=16384, k=1) == UNS and call(T=(1 << 22) - 1, H=256, k=1, wsb=16) == exm.ERR_WORKSPACE
    for name in AT:
        if name in ("residual", "logit_bias", "ws"):
            continue
        assert call(**{name: None}) == INV and name in exm.last_error()
        assert call(**{name: AT[name] + 8}) == INV and name in exm.last_error()
    assert call(ws=None) == exm.ERR_WORKSPACE == call(wsb=16)
    for out, other in (("y", "x"), ("y", "residual"), ("logits", "w_router"), ("topk_ids", "topk_weights"), ("residual", "x"), ("ws", "down"),
                       ("sorted_flat", "flat_to_sorted"), ("expert_offsets", "logit_bias")):
        assert call(**{out: AT[other]}) == INV and "overlaps" in exm.last_error(), (out, other)
    assert exm._lib.exmoe_moe_layer_fp8_workspace_bytes(4, 100, 128, 8, 2) == 0


def test_a_tensor_that_asks_for_a_gradient_is_refused():
    x = torch.ones((4, 256), dtype=BF16, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        exm.moe_layer_fp8(x, x, x, None, 2)


def test_experts_on_two_devices_are_refused():
    with pytest.raises(ValueError, match="same device"):
        exm.Fp8Experts(torch.ones((2, 256, 128)), torch.ones((2, 128, 128), device="meta"))


def operands(T, H, I, E, seed=0):
    gen = torch.Generator().manual_seed(seed + T)
    randn = lambda *s, sigma=1.0: torch.randn(s, generator=gen) * sigma  # noqa: E731
    x, res = randn(T, H).to(BF16).cuda(), randn(T, H, sigma=2.0).to(BF16).cuda()
    wn, wr = (1 + randn(H, sigma=0.1)).to(BF16).cuda(), randn(E, H, sigma=0.05).to(BF16).cuda()
    ex = exm.Fp8Experts(randn(E, 2 * I, H, sigma=0.05).cuda(), randn(E, H, I, sigma=0.05).cuda())
    return x, res, wn, wr, ex, randn(E, sigma=0.5).cuda()


def by_its_calls(x, res, wn, wr, ex, k, bias):
    n = exm.rms_norm(x, wn, residual=res, out="both")
    logits, ids, weights = exm.route_topk(n.y, wr, k, bias=bias)
    offsets, sorted_flat, f2s = exm.group_tokens(ids, ex.E)
    gate_up = exm.grouped_mm_fp8(n.q, n.scale, ex.gate_up, ex.gate_up_scale, offsets, row_index=sorted_flat, row_div=k)
    h, hs = exm.swiglu_fp8(gate_up, weights, sorted_flat)
    rows = exm.grouped_mm_fp8(h, hs, ex.down, ex.down_scale, offsets)
    y = torch.zeros((x.shape[0], x.shape[1]), device=x.device)
    for j in range(k):                                     # in slot order
        y += rows[f2s.view(-1, k)[:, j].long()].float()
    return dict(y=y.to(BF16), logits=logits, ids=ids, weights=weights, offsets=offsets, sorted_flat=sorted_flat, flat_to_sorted=f2s,
                residual=n.residual)


def same(b, want, res, label=""):
    for name, v in want.items():
        got = res if name == "residual" else getattr(b, name)
        assert v is None or torch.equal(got[:len(v)], v), f"{label}: {name}"


@gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (16, 2048, 1024, 16, 8), (100, 256, 384, 8, 3), (700, 512, 128, 12, 9), (2000, 256, 256, 4, 4)])
def test_the_layer_is_its_calls(T, H, I, E, k):
    x, res, wn, wr, ex, bias = operands(T, H, I, E)
    for with_res, with_bias in ((True, True), (False, False)):
        r = res.clone() if with_res else None
        want = by_its_calls(x, r, wn, wr, ex, k, bias if with_bias else None)
        b = exm.moe_layer_fp8(x, wn, wr, ex, k, residual=r, bias=bias if with_bias else None)
        same(b, want, r, f"residual {with_res}")


@gpu
@pytest.mark.parametrize("T", [1, 40])
def test_near_64_bits(T):
    """e4m3 activations twice: 4.7% of the result's norm (the derivation stands in test_fp8_experts.py)."""
    H, I, E, k = 256, 256, 8, 2
    x, res, wn, wr, ex, _ = operands(T, H, I, E)
    h = (x.float() + res.float()).to(BF16).double().cpu()
    b = exm.moe_layer_fp8(x, wn, wr, ex, k, residual=res)
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * wn.cpu().double()
    wide = lambda q, s: q.cpu().float().double() * s.cpu().double().repeat_interleave(128, 1).repeat_interleave(128, 2)  # noqa: E731
    gu, d = wide(ex.gate_up, ex.gate_up_scale), wide(ex.down, ex.down_scale)
    want = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            g, u = (gu[int(b.ids[t, j])] @ n[t]).split(I)
            want[t] += float(b.weights[t, j]) * (d[int(b.ids[t, j])] @ (g / (1 + torch.exp(-g)) * u))
    assert float((b.y.cpu().double() - want).norm() / want.norm()) < 0.06


@gpu
def test_captured_on_another_stream_and_empty():
    T, H, I, E, k = 30, 256, 128, 8, 2
    x, res, wn, wr, ex, bias = operands(T, H, I, E)
    first = res.clone()
    buffers = exm.Fp8LayerBuffers(T, H, I, E, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        exm.moe_layer_fp8(x, wn, wr, ex, k, residual=res, buffers=buffers)
    torch.cuda.current_stream().wait_stream(side)
    same(buffers, by_its_calls(x, first, wn, wr, ex, k, None), res, "stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        exm.moe_layer_fp8(x, wn, wr, ex, k, residual=res, buffers=buffers)
    for i in range(4):
        x.copy_(torch.randn((T, H)).to(BF16))
        before = res.clone()
        graph.replay()
        torch.cuda.synchronize()
        same(buffers, by_its_calls(x, before, wn, wr, ex, k, None), res, f"replay {i}")
    b = exm.moe_layer_fp8(x[:0], wn, wr, ex, k)
    assert b.offsets.tolist() == [0] * (E + 1) and b.y.shape == (0, H)
    for bad in (lambda: exm.moe_layer_fp8(x.float(), wn, wr, ex, k), lambda: exm.moe_layer_fp8(x, wn[:5], wr, ex, k),
                lambda: exm.moe_layer_fp8(x, wn, wr[:3], ex, k), lambda: exm.moe_layer_fp8(x, wn, wr, ex, k, residual=res[:3]),
                lambda: exm.moe_layer_fp8(x, wn, wr, ex, k + 1, buffers=buffers), lambda: exm.Fp8Experts(ex.gate_up_scale, ex.down_scale),
                lambda: exm.moe_layer_fp8(x, wn, wr, ex, k, bias=bias.double())):
        with pytest.raises(ValueError):
            bad()
