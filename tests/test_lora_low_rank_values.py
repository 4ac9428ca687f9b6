"""The adapters' v = A x between their two products: no bits of its 32 are lost on the way, in
every form of lora_linear, also where the 16 ranks that share a scale differ by powers of two.

W is zero, so that an output is the adapter's part alone: scale B v, rounded once.

Tolerances. v is off by ev = K 2^-23 |A||x| (an fp32 sum of K exact products; an adder that
drops the bits below loses at most 2^-23 of the running sum). v is passed on as four 16-bit
terms. bf16: three of them hold 24 bits, and 8 exponent bits are fp32's own, so nothing is
lost. fp16: the 16 ranks are scaled so that the largest lies in [2^14, 2^15); two terms hold a
value to 2^-25 or 2^-22 of it, two more, 2^23 times larger, hold the rest to 2^-25: 2^-48 in
all, 2^-62 of the largest. The sum over R ranks of four terms each: 4 R 2^-23 |B||v|. Scaling
rounds once more: 2^-23 of the result. The 16-bit output adds half a step, eps / 2 of its
value, at least eps / 2 of the smallest normal number."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16, FP16 = torch.bfloat16, torch.float16
gpu = pytest.mark.gpu

# (T, N, K, adapters, rank): one launch with one and with four blocks of ranks; 16 x 16, 32 x 32
# and 64 x 64 blocks; tiles of 128 x 128 and 256 x 256
FORMS = [(1, 40, 64, 1, 16), (9, 72, 64, 2, 32), (16, 200, 136, 6, 40), (70, 200, 136, 6, 40), (150, 700, 136, 6, 40),
         (150, 2604, 136, 6, 40), (601, 3804, 72, 6, 40), (4100, 4004, 64, 6, 16)]


def both_ways(x, b_n, bank, ids, dtype, K):
    """The adapter's part beside a W of zeros, and added to a y of zeros."""
    T = len(ids)
    idd, xd = ids.to(torch.int32).cuda(), x.to(dtype).cuda()
    yield "with w", exm.lora_linear(xd, torch.zeros((b_n, K), dtype=dtype, device="cuda"), bank, idd)
    y = torch.zeros((T, b_n), dtype=dtype, device="cuda")
    yield "added to y", exm.lora_linear(xd, None, bank, idd, y=y)


@gpu
@pytest.mark.parametrize("T,N,K,L,R", FORMS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_large_whole_numbers_cancel(T, N, K, L, R, dtype):
    """v of 20 (bf16) and 23 (fp16) bits, of which an output takes the difference of two ranks:
    every partial sum is a whole number below 2^24, so it is exact whatever the order."""
    print(f"cancel T={T} N={N} K={K} L={L} R={R} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(T + R)
    top, parts = (255, 15) if dtype is BF16 else (2047, 1)
    x = torch.zeros((T, K), dtype=torch.float64)
    x[:, :parts] = torch.randint(top // 2, top + 1, (T, parts), generator=gen).double()
    x[:, K - 1] = torch.randint(1, 3, (T,), generator=gen).double()
    a = torch.zeros((L, R, K), dtype=torch.float64)
    a[:, :, :parts] = torch.randint(top // 2, top + 1, (L, 1, parts), generator=gen).double()
    a[:, :, K - 1] = torch.randint(-20, 21, (L, R), generator=gen).double()
    plus = torch.stack([torch.randperm(R, generator=gen)[:2] for _ in range(N)])
    b = torch.zeros((L, N, R), dtype=torch.float64)
    b[:, torch.arange(N), plus[:, 0]], b[:, torch.arange(N), plus[:, 1]] = 1.0, -1.0
    ids = torch.randint(0, L, (T,), generator=gen)
    v = torch.einsum("tk,trk->tr", x, a[ids])
    assert v.abs().max() < 2 ** 23 and v.abs().max() >= 2 ** (18 if dtype is BF16 else 20)
    ref = (v[:, plus[:, 0]] - v[:, plus[:, 1]]).to(dtype)
    bank = exm.LoraBank(a.to(dtype).cuda(), b.to(dtype).cuda())
    for label, y in both_ways(x, N, bank, ids, dtype, K):
        wrong = y.cpu() != ref
        assert not wrong.any(), f"{label}: {int(wrong.sum())} of {wrong.numel()} differ"


@gpu
@pytest.mark.parametrize("T,N,K,L,R", FORMS)
@pytest.mark.parametrize("dtype,apart", [(FP16, 12), (FP16, 24), (FP16, 30), (FP16, 36), (BF16, 24), (BF16, 60)])
def test_ranks_of_different_sizes_share_a_block(T, N, K, L, R, dtype, apart):
    """In each block of 16 ranks one v is about 2^apart times the others, and B does not use it."""
    print(f"apart 2^{apart} T={T} N={N} K={K} L={L} R={R} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(T + R + apart)
    low = max(-apart, -22) if dtype is FP16 else -apart // 2      # exponent of the small rows of A
    x = torch.randn((T, K), generator=gen).to(dtype).double()
    a = (torch.randn((L, R, K), generator=gen) * 2.0 ** low).to(dtype).double()
    big = torch.arange(0, R, 16) + torch.tensor([3, 0, 7])[:len(range(0, R, 16))]
    a[:, big] = (torch.randn((L, len(big), K), generator=gen).clamp(-3, 3) * 2.0 ** (apart + low)).to(dtype).double()
    assert a.isfinite().all()
    b = torch.randn((L, N, R), generator=gen) * 2.0 ** min(12, -low)
    b[:, :, big] = 0.0
    b = b.to(dtype).double()
    scales = torch.rand(L, generator=gen) + 0.5
    ids = torch.randint(0, L, (T,), generator=gen)
    v = torch.einsum("tk,trk->tr", x, a[ids])
    ref, bound = torch.empty((T, N), dtype=torch.float64), torch.empty((T, N), dtype=torch.float64)
    ev = torch.einsum("tk,trk->tr", x.abs(), a[ids].abs()) * K * 2.0 ** -23
    eh = 2.0 ** -62 * v.abs().amax(1, keepdim=True) if dtype is FP16 else 0.0
    for i in range(L):
        t, s, B = ids == i, float(scales[i]), b[i]
        ref[t] = s * (v[t] @ B.t())
        bound[t] = s * ((ev + eh)[t] + 4 * R * 2.0 ** -23 * v[t].abs()) @ B.abs().t() + 2.0 ** -23 * ref[t].abs()
    fi = torch.finfo(dtype)
    assert ref.abs().max() < fi.max
    bound = bound + fi.eps / 2 * (ref.abs() + bound).clamp(min=fi.tiny)
    bank = exm.LoraBank(a.to(dtype).cuda(), b.to(dtype).cuda(), scales=scales.float().cuda())
    for label, y in both_ways(x, N, bank, ids, dtype, K):
        off = (y.cpu().double() - ref).abs()
        bad = ~(off <= bound)
        assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {float((off / bound).max()):.1f} of it"
