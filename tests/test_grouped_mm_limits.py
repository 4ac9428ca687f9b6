"""Sizes near the limits of a launch: what fits in some form runs, what fits in none is refused
before anything is enqueued. Whole numbers, so results are equal bit for bit."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16, FP32 = torch.bfloat16, torch.float32
FAKE = 0x10000
gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("N,offset", [(493608, 1), (986912, 0)])
def test_few_rows_of_many_wide_experts(N, offset):
    """One row for each of 256 experts: more 16 x 16 blocks than a launch holds (512 threads each
    where rows are not 16-byte aligned, else 256), few 128 x 128 tiles."""
    print(f"wide N={N} offset={offset}", flush=True)
    E, K = 256, 8
    assert (E // 16 + E) * ((N + 15) // 16) * (512 if offset else 256) > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randint(-2, 3, (E, K), generator=gen, device="cuda").to(BF16)
    buf = torch.empty(E * N * K + offset, dtype=BF16, device="cuda")
    w = buf[offset:].view(E, N, K)
    for e in range(E):
        w[e] = torch.randint(-2, 3, (N, K), generator=gen, device="cuda").to(BF16)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    y = exm.grouped_mm(x, w, off)
    for e in range(E):
        ref = (w[e].float() * x[e].float()).sum(1)
        assert torch.equal(y[e], ref.to(BF16)), f"expert {e}"


def test_copies_that_fit_no_launch_are_refused_first():
    """Operands with odd row lengths whose copy needs more threads than a launch has, beside a
    product that fits: refused (the pointers are never followed)."""
    rows, K, N = 1 << 24, 2049, 64
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_MM, rows, N, K, 1)
    st = exm._lib.exmoe_grouped_mm(FAKE, K, rows, None, 1, 1 << 52, 1 << 51, K, N * K, rows, N, K, 1, 0, 0, 1 << 50, N,
                                   1 << 48, need, None)
    assert st == exm.ERR_UNSUPPORTED and "launch" in exm.last_error()
    need = exm.grouped_mm_workspace_bytes(exm.GROUPED_WGRAD, rows, K, 8, 1)
    st = exm._lib.exmoe_grouped_mm_wgrad(FAKE, K, 1 << 52, 8, rows, None, 1, 1 << 51, rows, K, 8, 1, 0, 2, 1 << 50, 8,
                                         8 * K, 1 << 48, need, None)
    assert st == exm.ERR_UNSUPPORTED and "launch" in exm.last_error()


def test_token_sums_of_four_columns_a_thread():
    """Sums over 2^20 tokens of 8192 columns are 2^31 threads, of 8191 columns 2^33 less 2^20: the
    size is looked at before the workspace, which is missing here."""
    def call(K):
        return exm._lib.exmoe_grouped_mm_dgrad(FAKE, 64, 1 << 52, 1 << 51, K, 64 * K, 1 << 49, 2, 1 << 21, 64, K, 1, 0, 0,
                                               1 << 50, K, None, 0, None)
    assert call(8192) == exm.ERR_WORKSPACE
    assert call(8191) == exm.ERR_UNSUPPORTED
