"""The router's losses over the longest batch: the sums over tokens against 64 bits.

Equal rows, so that every addition of a running sum rounds the same way: 2048 additions of a probability in 32
bits, one after another, are off by up to 2.9e-5 of their sum (for the rows below). Tolerance: a probability is
off by 2^-18 of itself and a log-sum-exp by 2^-18 (the derivation stands in test_balance_loss.py); a lane adds 16
rows in 32 bits and those sums in 64, rounds once, the result is added to those of at most 2 rows of lanes and 16
waves, and the loss is rounded once: under 40 roundings of 2^-24, 2^-18 in all."""
import pytest

exm = pytest.importorskip("w4a16_mixture_experts_amd")
torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu


@gpu
def test_equal_rows_of_the_longest_batch():
    T, E = 1 << 24, 129                  # 2048 rows a lane
    row = (torch.randn(E, generator=torch.Generator().manual_seed(11)) * 1.5).to(torch.bfloat16)
    lse = torch.logsumexp(row.double(), 0)
    p = torch.exp(row.double() - lse)
    logits = row.cuda().expand(T, E).contiguous()
    ids, ws = torch.empty((T, 1), dtype=torch.int32, device="cuda"), exm.alloc_workspace(exm.balance_loss_workspace_bytes(T, E))
    for e in range(0, E, 8):             # every token routed to e: E p_e
        ids.fill_(e)
        losses, counts = exm.balance_loss(logits, ids, workspace=ws)
        balance, z = losses.tolist()
        assert int(counts[e]) == T == int(counts[E]) and int(counts.sum()) == 2 * T
        off = abs(balance / (E * float(p[e])) - 1)
        assert off <= 2.0 ** -18 + 2.0 ** -18, f"balance with expert {e}: {off:.2e}"
        off = abs(z - float(lse ** 2))
        assert off <= 2.0 ** -17 * float(lse) + 2.0 ** -36 + 2.0 ** -18 * float(lse ** 2), f"z: off by {off:.2e}"
