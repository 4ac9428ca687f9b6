"""Adapters beside a projection at sizes near a launch's limit: many tokens times many columns."""
import ctypes

import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

BF16 = torch.bfloat16
gpu = pytest.mark.gpu


def status(T, N, w=True):
    """The refusal of a call whose workspace is missing: its size's, or the workspace's."""
    far = [i << 44 for i in range(1, 9)]
    bank = exm.LoraBankC(far[0], 64, 64 * 16, far[1], 16, N * 16, None, None, 3, 16)
    return exm._lib.exmoe_lora_linear(far[2], 64, far[3] if w else None, 64, ctypes.byref(bank), far[4], T, N, 64, 0, far[5], N,
                                      None, 0, None)


def test_sizes():
    for T, N in ((131072, 16384), (1 << 20, 65000), (1 << 22, 16000), (65000, 1 << 20)):
        for w in (True, False):
            assert status(T, N, w) == exm.ERR_WORKSPACE, (T, N)
            assert exm.lora_workspace_bytes(T, N, 64, 3, 16) > 0
    for T, N in ((1 << 20, 1 << 17), (1 << 22, 1 << 20)):          # 2^37 outputs and more: 2^33 threads
        assert status(T, N) == exm.ERR_UNSUPPORTED and exm.lora_workspace_bytes(T, N, 64, 3, 16) == 0


@gpu
@pytest.mark.parametrize("T,N", [(131072, 16384), (200000, 12001)])
def test_many_tokens_times_many_columns(T, N):
    """More than 2^31 outputs, beside W and added to y."""
    print(f"large T={T} N={N}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(N)
    K, L, R = 8, 3, 8

    def whole(*s):
        return torch.randint(-1, 2, s, generator=gen, device="cuda").to(BF16)

    x, w, bank = whole(T, K), whole(N, K), exm.LoraBank(whole(L, R, K), whole(L, N, R))
    ids = torch.randint(-1, L, (T,), generator=gen, device="cuda", dtype=torch.int32)

    def part(t):                                              # the adapters' part of some tokens, whole numbers
        d = torch.zeros((len(t), N), device="cuda")
        for i in range(L):
            d += (ids[t] == i).unsqueeze(1).float() * ((x[t].float() @ bank.a[i].float().t()) @ bank.b[i].float().t())
        return d

    some = torch.cat([torch.arange(512), torch.arange(T // 2 - 256, T // 2 + 256), torch.arange(T - 512, T)]).cuda()
    y = exm.lora_linear(x, w, bank, ids)
    assert torch.equal(y[some], (x[some].float() @ w.float().t() + part(some)).to(BF16))
    y.fill_(1.0)
    exm.lora_linear(x, None, bank, ids, y=y)
    assert torch.equal(y[some], (1.0 + part(some)).to(BF16))
    sums = torch.cat([c.float().sum(1) for c in y.split(8192)])
    assert bool((sums[ids < 0] == N).all()), "a token without an adapter changed"
