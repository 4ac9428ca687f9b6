"""The expert layer in 8 bits on batches whose products run on the large tiles: bit for bit what its calls give one by
one, repeated, and near the layer whose rows stay in 32 bits."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

from test_fp8_tile_forms import form  # noqa: E402
from test_layer_fp8 import BF16, by_its_calls, operands, same  # noqa: E402

gpu = pytest.mark.gpu
# T, H, I, E, k and the forms of gate and up and of down
PROMPTS = [(400, 512, 1280, 16, 4, (128, 128), (16, 64, 2)), (4096, 1024, 512, 4, 4, (192, 256), (192, 256)), (2048, 256, 3200, 1, 1, (256, 256), (16, 64, 2))]


def test_the_listed_sizes_reach_their_forms():
    for T, H, I, E, k, up, down in PROMPTS:
        assert (form(T * k, E, 2 * I, H, BF16), form(T * k, E, H, I, BF16)) == (up, down), (T, H, I, E, k)


@gpu
@pytest.mark.parametrize("T,H,I,E,k,up,down", PROMPTS)
def test_the_layer_is_its_calls(T, H, I, E, k, up, down):
    x, res, wn, wr, ex, bias = operands(T, H, I, E)
    before = res.clone()
    want = by_its_calls(x, before, wn, wr, ex, k, bias)
    for _ in range(3):
        r = before.clone()
        same(exm.moe_layer_fp8(x, wn, wr, ex, k, residual=r, bias=bias), want, r)


@gpu
@pytest.mark.parametrize("T,H,I,E,k,up,down", PROMPTS)
def test_what_rows_in_16_bits_cost(T, H, I, E, k, up, down):
    """Down rows rounded to bf16 before their sum, against the separate calls with rows in 32 bits. A rounding is off
    by at most 2^-8 of its value, 0.43 of that on average over a power of two (its square's mean: a third, of values
    1 to 2), so 2^-8 of the norms of the rows and of y leaves more than half for what the 16-bit product loses beside
    them (1.6e-5 of its norm)."""
    x, _, wn, wr, ex, bias = operands(T, H, I, E)
    b = exm.moe_layer_fp8(x, wn, wr, ex, k, bias=bias)
    n = exm.rms_norm(x, wn, out="fp8")
    gate_up = exm.grouped_mm_fp8(n.q, n.scale, ex.gate_up, ex.gate_up_scale, b.offsets, row_index=b.sorted_flat, row_div=k)
    h, hs = exm.swiglu_fp8(gate_up, b.weights, b.sorted_flat)
    rows = exm.grouped_mm_fp8(h, hs, ex.down, ex.down_scale, b.offsets, out_dtype=torch.float32)
    by_token = rows[b.flat_to_sorted.long()].view(T, k, H).double()
    want, norm = by_token.sum(1), float(by_token.sum(1).norm())
    off = float((b.y.double() - want).norm())
    assert off <= 2.0 ** -8 * (float(by_token.square().sum(1).sqrt().norm()) + norm), off / norm
