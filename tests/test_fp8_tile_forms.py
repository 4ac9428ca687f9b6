"""The 8-bit product on each of the forms that its rule chooses: several slices of the summed axis, odd and even in
number, the last one cut; full and partly filled tiles; normal values, whole numbers, NaN, repeated calls.

A slice is 128 positions, and the tiles keep two of them in LDS in turn: from the third on a slice is copied over an
earlier one. form() is the rule written once more, so that a size which no longer reaches the form it is listed for
fails here instead of testing another one.

Tolerances: product_bound() of test_fp8_experts.py; sums of whole numbers are exact."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

from test_fp8_experts import BF16, F8, FP16, FP32, offsets_of, on_gpu, product_bound, spread  # noqa: E402

gpu = pytest.mark.gpu


def form(rows, E, N, K, dtype):
    """The rows x columns of a tile, and for the blocks of few rows their waves."""
    used, cols = min(E, rows), lambda q: -(-N // q)
    tiles = (rows // 128 + used) * cols(128)

    def few_blocks(bq):
        return K >= 2048 and (rows // 16 + used) * cols(bq) <= 384

    if rows <= 12 * E:
        return (16, 32, 4 if K >= 4096 or few_blocks(32) else 2)
    if tiles < 128:
        return (16, 64, 4 if few_blocks(64) else 2)
    if tiles < 512 or rows <= 48 * E:
        return (64, 128)
    if dtype is not FP32 and rows // E >= 160 and rows // 256 * cols(256) >= 200:
        def rounds(bp):
            if E > 1:
                return (rows / bp + 0.5 * used) * cols(256) / 256 + 0.5
            return -(-(-(-rows // bp) * cols(256)) // 256)
        return (192, 256) if 0.8 * rounds(192) < rounds(256) else (256, 256)
    return (128, 128)


# counts per expert, N, and the form in 16 bits and in 32
FORMS = [([2, 0, 9, 1], 200, (16, 32, 2), (16, 32, 2)), ([100, 30, 7], 264, (16, 64, 2), (16, 64, 2)), ([300, 40, 170], 5000, (64, 128), (64, 128)),
         ([90, 0, 130, 77] * 4, 4100, (128, 128), (128, 128)), ([128] * 16, 2560, (128, 128), (128, 128)),
         ([1200, 3, 900], 6700, (192, 256), (128, 128)), ([960, 3, 960], 7700, (192, 256), (128, 128)),
         ([2049], 6400, (256, 256), (128, 128)), ([2048], 6400, (256, 256), (128, 128))]
DEPTHS = [656, 784]                       # 5.1 and 6.1 slices
LONG = [([3, 0, 5], 264, 2320, (16, 32, 4)), ([1, 0, 2], 264, 4112, (16, 32, 4)), ([100, 2, 30], 264, 2320, (16, 64, 4))]
EVERY = [(c, N, K, f16, f32) for c, N, f16, f32 in FORMS for K in DEPTHS] + [(c, N, K, f, f) for c, N, K, f in LONG]


def test_the_listed_sizes_reach_their_forms():
    for counts, N, K, f16, f32 in EVERY:
        for dtype, want in ((BF16, f16), (FP16, f16), (FP32, f32)):
            assert form(sum(counts), len(counts), N, K, dtype) == want, (counts, N, K, dtype)
    assert {f for _, _, _, f, _ in EVERY} == {(16, 32, 2), (16, 32, 4), (16, 64, 2), (16, 64, 4), (64, 128), (128, 128), (192, 256), (256, 256)}


def seeded(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return gen, lambda *shape: torch.randn(shape, generator=gen, device="cuda")


def whole_operands(gen, rows, E, N, K):
    """Small whole numbers and scales of powers of two: sums are exact."""
    def pick(values, *shape):
        return torch.tensor(values, device="cuda")[torch.randint(0, 5, shape, generator=gen, device="cuda")]
    kb, nb = (K + 127) // 128, (N + 127) // 128
    ints, powers = [-2.0, -1.0, 0.0, 1.0, 2.0], [0.25, 0.5, 1.0, 2.0, 4.0]
    return pick(ints, rows, K).to(F8), pick(powers, rows, kb), pick(ints, E, N, K).to(F8), pick(powers, E, nb, kb)


def reference(x, xs, w, ws, counts, src, cuts=False):
    """y, the products' magnitudes and the largest product of each 8 neighbours, summed, in 64 bits on the GPU."""
    E, N, K = w.shape
    xr = (x.float() * spread(xs, x.shape[0], K))[src.clamp(min=0)] * (src >= 0)[:, None]
    y, mag, cut = (torch.zeros((len(src), N), dtype=torch.float64, device="cuda") for _ in range(3))
    at = 0
    for e, n in enumerate(counts):
        a, b, at = at, at + n, at + n
        if not n:
            continue
        # (q x scale is exact in 64 bits, not in 32)
        xe = (x.double() * spread(xs.double(), x.shape[0], K))[src[a:b].clamp(min=0)] * (src[a:b] >= 0)[:, None]
        we = w[e].double() * spread(ws[e].double(), N, K, 128)
        y[a:b] = xe @ we.t().contiguous()
        if cuts:
            mag[a:b] = xe.abs() @ we.abs().t().contiguous()
            xa, wa = xr[a:b].abs(), we.abs().float()
            for k in range(0, K, 8):
                top = xa[:, k, None] * wa[None, :, k]
                for j in range(k + 1, k + 8):
                    top = torch.maximum(top, xa[:, j, None] * wa[None, :, j])
                cut[a:b] += top
    return y, mag, cut


def gathered(gen, rows, k):
    """Tokens' slots in any order, one without a row of x and one past its end."""
    T = rows // k + 3
    index = torch.randint(0, T * k, (rows,), generator=gen, device="cuda").to(torch.int32)
    index[0] = -1
    index[-1] = T * k + 7
    src = torch.where(index >= 0, index // k, -1).long()
    return T, index, torch.where(src < T, src, -1)


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("counts,N,K,f16,f32", EVERY)
def test_normal_values(counts, N, K, f16, f32, dtype):
    gen, randn = seeded(N + K)
    rows, k = sum(counts), 2
    T, index, src = gathered(gen, rows, k)
    x8, xs = exm.quantize_fp8(randn(T, K))
    w8, ws = exm.quantize_fp8_weights(0.02 * randn(len(counts), N, K))
    off = offsets_of(counts).cuda()
    call = lambda: exm.grouped_mm_fp8(x8, xs, w8, ws, off, row_index=index, row_div=k, out_dtype=dtype)  # noqa: E731
    got = call()
    y, mag, cut = reference(x8, xs, w8, ws, counts, src, cuts=dtype is not FP32)
    if dtype is FP32:
        mag = reference(x8.float().abs(), xs, w8.float().abs(), ws, counts, src)[0]
    bad = ~((got.double() - y).abs() <= product_bound(y, mag, cut, K, dtype))
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:4].tolist()}"
    for _ in range(3):
        assert torch.equal(call().view(torch.uint8), got.view(torch.uint8))


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("counts,N,K,f16,f32", EVERY)
def test_whole_numbers(counts, N, K, f16, f32, dtype):
    """Rows of x in order, longer than K with NaN behind it; y inside a wider matrix, whose other columns stay."""
    gen, _ = seeded(N + K + 1)
    rows = sum(counts)
    x, xs, w, ws = whole_operands(gen, rows, len(counts), N, K)
    y, _, _ = reference(x, xs, w, ws, counts, torch.arange(rows, device="cuda"))
    for left, more in ((0, 0), (1, 3)):
        out = torch.full((rows, N + more), 7.0, dtype=dtype, device="cuda")
        exm.grouped_mm_fp8(on_gpu(x, 0, 16), xs, on_gpu(w, 0, 16), ws, offsets_of(counts).cuda(), y=out[:, left:left + N], out_dtype=dtype)
        assert torch.equal(out[:, left:left + N], y.to(dtype)), f"{int((out[:, left:left + N] != y.to(dtype)).sum())} differ"
        out[:, left:left + N] = 7.0
        assert bool((out == 7).all())


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("counts,N,K,f16,f32", [c for c in EVERY if max(c[0]) > 4])
def test_a_nan_stays_in_its_row_and_column(counts, N, K, f16, f32, dtype):
    """In the last, cut slice of a row and of a column, and in a scale of each."""
    gen, _ = seeded(N + K + 2)
    rows, e = sum(counts), max(range(len(counts)), key=lambda i: counts[i])
    first = sum(counts[:e])
    x, xs, w, ws = whole_operands(gen, rows, len(counts), N, K)
    y, _, _ = reference(x, xs, w, ws, counts, torch.arange(rows, device="cuda"))
    xf, wf = x.float(), w.float()
    xf[first + 1, K - 2], wf[e, 40, K - 9] = float("nan"), float("nan")
    xs[first + 3, 1], ws[e, 1, 2] = float("inf"), float("nan")          # (the latter: columns 128 to 255)
    got = exm.grouped_mm_fp8(xf.to(F8), xs, wf.to(F8), ws, offsets_of(counts).cuda(), out_dtype=dtype)
    seg = slice(first, first + counts[e])
    nan = torch.zeros((rows, N), dtype=torch.bool, device="cuda")
    nan[first + 1], nan[seg, 40], nan[seg, 128:256] = True, True, True
    assert bool(torch.isnan(got[nan]).all()) and not bool(torch.isfinite(got[first + 3]).any())
    nan[first + 3] = True
    assert torch.equal(got[~nan], y.to(dtype)[~nan])
