"""Cases of the 8-bit expert path's operators and of the router's balance loss: inputs, the calls
and their plain form.

Operators (in `kind`). 8-bit values are e4m3; a scale s stands for 128 neighbours of a row (of a
128 x 128 block of a weight matrix): value = q s, s = largest |value| of the block / 448.
  norm         h = round(x + residual); y = h / sqrt(mean(h^2) + eps) * w, in 16 bits and as (q, s)
  act          a = silu(gate) * up of each routed row as (q, s), s times the row's routing weight;
               or a matrix as (q, s) as it is
  mm           y[s, :] = W_e x[src(s), :], both in 8 bits; rows gathered from the tokens, grouped by
               expert (offsets[e]..offsets[e + 1]), or one matrix for all rows
  balance      of the M tokens that count: counts c_e of the routed pairs, balance
               E sum_e c_e / (M k) mean_t p_te, and z = mean_t (log sum_e exp l_te)^2, p = softmax(l)
  balance_bwd  their gradient with respect to the logits l
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_F8 = torch.float8_e4m3fn
_B = 128                          # values of one scale
_LEAST = 2.0 ** -126              # smallest scale


def _norm(name, T, H, dtype, residual, out):
    return {"name": name, "kind": "norm", "T": T, "H": H, "dtype": dtype, "residual": residual, "out": out}


def _act(name, rows, I, dtype, gated):
    return {"name": name, "kind": "act", "rows": rows, "I": I, "dtype": dtype, "gated": gated}


def _mm(name, T, k, E, N, K, out, zipf, gather):
    return {"name": name, "kind": "mm", "T": T, "k": k, "E": E, "N": N, "K": K, "out": out, "zipf": zipf, "gather": gather}


def _balance(name, kind, T, k, E, dtype, out, padded):
    return {"name": name, "kind": kind, "T": T, "k": k, "E": E, "dtype": dtype, "out": out, "padded": padded}


def listed():
    return [
        # one token's norm in front of the router (16 bits) and the experts (8 bits): latency
        _norm("norm_decode_1", 1, 2048, "bf16", "bf16", "both"),
        # rows that no vector load divides, a residual stream in 32 bits
        _norm("norm_odd", 389, 1003, "fp16", "fp32", "both"),
        # the large layer's norm over a prompt of 4096 tokens: bandwidth
        _norm("norm_prefill_4096", 4096, 4096, "bf16", "bf16", "both"),
        # the hidden rows of a decode batch of 16 tokens with 8 experts each: latency
        _act("act_decode_16", 128, 1024, "bf16", True),
        # the hidden rows of a prompt of 2048 tokens: bandwidth
        _act("act_prefill_2048", 16384, 1024, "bf16", True),
        # the tiny layer's gate and up rows, 16 tokens, two experts a token: latency
        _mm("mm_tiny", 16, 2, 8, 512, 256, "bf16", False, True),
        # gate and up of a decode batch of 16 tokens: bandwidth of the 8-bit weights
        _mm("mm_decode_16", 16, 8, 64, 2048, 2048, "bf16", False, True),
        # a prompt of 2048 tokens with skewed experts, some of them empty
        _mm("mm_zipf_2048", 2048, 8, 64, 2048, 2048, "bf16", True, True),
        # sizes that no tile divides; the last block of rows, columns and summed positions is cut
        _mm("mm_odd", 389, 2, 13, 517, 1008, "fp32", False, True),
        # the large experts' up projection over 4096 tokens: matrix rate
        _mm("mm_large", 4096, 2, 8, 14336, 4096, "bf16", False, True),
        # the router's losses over a padded batch of prompts
        _balance("balance_8192", "balance", 8192, 8, 64, "bf16", "bf16", True),
        # their gradient over a long training batch, in 32 bits
        _balance("balance_bwd_65536", "balance_bwd", 65536, 8, 128, "fp32", "fp32", False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    """Half of the sizes in whole blocks, the others ragged (multiples of `step`)."""
    n = _log_int(rng, lo, hi)
    if rng.random() < 0.5:
        return max(_B, (n + _B // 2) // _B * _B)
    return max(step, n // step * step) if step > 1 else n | 1


def draw(rng):
    kind = rng.choice(["norm", "norm", "act", "mm", "mm", "mm", "balance", "balance_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    while True:
        if kind == "norm":
            T, H = _log_int(rng, 1, 16384), _size(rng, 64, 16384, 1)
            if T * H > 4 * 4096 * 4096:
                continue
            return {"kind": kind, "T": T, "H": H, "dtype": dtype, "residual": rng.choice(["none", dtype, "fp32"]),
                    "out": rng.choice(["y", "fp8", "both"])}
        if kind == "act":
            rows, I = _log_int(rng, 1, 32768), _size(rng, 64, 14336, 1)
            if rows * I > 2 * 16384 * 1024:
                continue
            return {"kind": kind, "rows": rows, "I": I, "dtype": dtype, "gated": rng.random() < 0.7}
        T = _log_int(rng, 1, 4096)
        E = rng.choice([1, _log_int(rng, 1, 128), _log_int(rng, 4, 128)])
        k = rng.choice([j for j in (1, 2, 4, 6, 8) if j <= E])
        if kind == "mm":
            N, K = _size(rng, 64, 14336, 1), _size(rng, 64, 8192, 16)
            if E * N * K > 8 * 14336 * 4096 or T * k * N * K > 8192 * 14336 * 4096 or T * k > 16384:
                continue
            return {"kind": kind, "T": T, "k": k, "E": E, "N": N, "K": K, "out": rng.choice(["bf16", "fp16", "fp32"]),
                    "zipf": rng.random() < 0.5, "gather": rng.random() < 0.5}
        return {"kind": kind, "T": _log_int(rng, 1, 65536), "k": k, "E": E, "dtype": dtype,
                "out": rng.choice([dtype, "fp32"]), "padded": rng.random() < 0.5}


# ------------------------------------------------------------------------------------ inputs
def _quantized(v, rows):
    """fp32 [..., n, K] as e4m3 values and scales of blocks of `rows` x 128."""
    n, K = v.shape[-2:]
    pn, pk = -n % rows, -K % _B
    p = torch.nn.functional.pad(v, (0, pk, 0, pn))
    p = p.view(*v.shape[:-2], (n + pn) // rows, rows, (K + pk) // _B, _B)
    scale = (p.abs().amax(dim=(-3, -1)) / 448.0).clamp(min=_LEAST)
    q = (p / scale[..., :, None, :, None]).to(_F8).view(*v.shape[:-2], n + pn, K + pk)
    return q[..., :n, :K].contiguous(), scale


def _rows_by_expert(case, gen):
    """Offsets and order of routed pairs (token, slot), sorted by expert: the k largest of noisy
    logits, skewed by the experts' popularity under zipf."""
    T, k, E = case["T"], case["k"], case["E"]
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    if case["zipf"]:
        noise = noise - 1.1 * torch.log(torch.randperm(E, generator=gen, device="cuda") + 1.0)
    flat = torch.topk(noise, k, dim=1).indices.reshape(-1)
    ids, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(ids, torch.arange(E + 1, device="cuda"))
    return offsets.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 41)

    def randn(*shape, sigma=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * sigma

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    kind = case["kind"]
    st = dict(case)
    if kind == "norm":
        T, H, dt = case["T"], case["H"], _TYPES[case["dtype"]]
        st.update(x=randn(T, H).to(dt), w=(1.0 + randn(H, sigma=0.1)).to(dt), eps=1e-6, res=None)
        if case["residual"] != "none":
            st["res"] = randn(T, H, sigma=2.0).to(_TYPES[case["residual"]])
        if own:
            st["o"] = {}
            if case["out"] != "fp8":
                st["o"]["y"] = empty(T, H, dtype=dt)
            if case["out"] != "y":
                st["o"].update(q=empty(T, H, dtype=_F8), scale=empty(T, -(-H // _B), dtype=torch.float32))
            if st["res"] is not None:
                st["o"]["residual_out"] = torch.empty_like(st["res"])
    elif kind == "act":
        rows, I, dt = case["rows"], case["I"], _TYPES[case["dtype"]]
        st["x"] = randn(rows, 2 * I if case["gated"] else I, sigma=1.5).to(dt)
        if case["gated"]:
            st["weights"] = torch.rand(rows, generator=gen, device="cuda")
            st["order"] = torch.randperm(rows, generator=gen, device="cuda").to(torch.int32)
        if own:
            st["o"] = dict(q=empty(rows, I, dtype=_F8), scale=empty(rows, -(-I // _B), dtype=torch.float32))
    elif kind == "mm":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        st["offsets"], st["order"] = _rows_by_expert(case, gen)
        st["x"], st["xs"] = _quantized(randn(T if case["gather"] else T * k, K), 1)
        st["w"], st["ws"] = empty(E, N, K, dtype=_F8), empty(E, -(-N // _B), -(-K // _B), dtype=torch.float32)
        for e in range(E):                     # (one expert at a time: the 32-bit copies are large)
            st["w"][e], st["ws"][e] = _quantized(randn(N, K, sigma=0.02), _B)
        if own:
            st["y"] = empty(T * k, N, dtype=_TYPES[case["out"]])
        else:
            st["edges"] = st["offsets"].tolist()
    else:
        T, k, E = case["T"], case["k"], case["E"]
        st["l"] = randn(T, E, sigma=1.5).add_(randn(E)).to(_TYPES[case["dtype"]])
        st["ids"] = torch.topk(st["l"].float(), k, dim=1).indices.to(torch.int32)
        st["mask"] = None
        if case["padded"]:                     # prompts of different lengths, padded at their ends
            length = torch.randint(0, 257, (-(-T // 256),), generator=gen, device="cuda").clamp(min=1)
            st["mask"] = (torch.arange(256, device="cuda") < length[:, None]).reshape(-1)[:T].contiguous()
        if kind == "balance_bwd":
            live = st["ids"] if st["mask"] is None else st["ids"][st["mask"]]
            tokens = T if st["mask"] is None else int(st["mask"].sum())
            st["counts"] = torch.cat([torch.bincount(live.reshape(-1).long(), minlength=E),
                                      torch.tensor([tokens], device="cuda")]).to(torch.int32)
            st["dl"] = randn(2, sigma=0.01)
        if own:
            if kind == "balance":
                st["o"] = dict(losses=empty(2, dtype=torch.float32), counts=empty(E + 1, dtype=torch.int32))
            else:
                st["o"] = dict(dlogits=empty(T, E, dtype=_TYPES[case["out"]]))
    if own:
        import w4a16_mixture_experts_amd as exm
        st["exm"] = exm
        if kind == "balance":
            st["o"]["workspace"] = exm.alloc_workspace(exm.balance_loss_workspace_bytes(case["T"], case["E"]))
    return st


# ------------------------------------------------------------------------------------ one pass
def _run_own(st):
    exm, kind = st["exm"], st["kind"]
    if kind == "norm":
        r = exm.rms_norm(st["x"], st["w"], st["eps"], residual=st["res"], out=st["out"], **st["o"])
        return {n: v for n, v in (("y", r.y), ("q", r.q), ("scale", r.scale), ("residual", r.residual)) if v is not None}
    if kind == "act":
        if st["gated"]:
            q, scale = exm.swiglu_fp8(st["x"], weights=st["weights"], row_index=st["order"], **st["o"])
        else:
            q, scale = exm.quantize_fp8(st["x"], **st["o"])
        return {"q": q, "scale": scale}
    if kind == "mm":
        if st["E"] == 1 and not st["gather"]:
            return exm.grouped_mm_fp8(st["x"], st["xs"], st["w"], st["ws"], y=st["y"], out_dtype=st["y"].dtype)
        return exm.grouped_mm_fp8(st["x"], st["xs"], st["w"], st["ws"], st["offsets"],
                                  row_index=st["order"] if st["gather"] else None, row_div=st["k"], y=st["y"],
                                  out_dtype=st["y"].dtype)
    if kind == "balance":
        losses, counts = exm.balance_loss(st["l"], st["ids"], mask=st["mask"], **st["o"])
        return {"losses": losses, "counts": counts}
    return exm.balance_loss_backward(st["l"], st["counts"], st["k"], st["dl"], mask=st["mask"], out_dtype=_TYPES[st["out"]],
                                     **st["o"])


def _spread(scale, n):
    """Each scale in front of its 128 neighbours of the last axis, n of them in all."""
    return scale.repeat_interleave(_B, dim=-1)[..., :n]


def _as_fp8(v):
    K = v.shape[-1]
    blocks = torch.nn.functional.pad(v, (0, -K % _B)).view(v.shape[0], -1, _B)
    scale = (blocks.abs().amax(-1) / 448.0).clamp(min=_LEAST)
    return (v / _spread(scale, K)).to(_F8), scale


def _run_plain(st):
    kind = st["kind"]
    if kind == "norm":
        out, h = {}, st["x"].float()
        if st["res"] is not None:
            out["residual"] = (h + st["res"].float()).to(st["res"].dtype)
            h = out["residual"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + st["eps"]) * st["w"].float()
        if st["out"] != "fp8":
            out["y"] = y.to(st["x"].dtype)
        if st["out"] != "y":
            out["q"], out["scale"] = _as_fp8(y)
        return out
    if kind == "act":
        v = st["x"].float()
        if not st["gated"]:
            q, scale = _as_fp8(v)
            return {"q": q, "scale": scale}
        g, u = v[:, :st["I"]], v[:, st["I"]:]
        q, scale = _as_fp8(g / (1.0 + torch.exp(-g)) * u)
        return {"q": q, "scale": scale * st["weights"][st["order"].long()].unsqueeze(1)}
    if kind == "mm":
        x = st["x"].float() * _spread(st["xs"], st["K"])
        if st["gather"]:
            x = x[(st["order"] // st["k"]).long()]
        y = torch.empty((x.shape[0], st["N"]), dtype=torch.float32, device="cuda")
        for e, (a, b) in enumerate(zip(st["edges"], st["edges"][1:])):
            if a < b:
                s = _spread(st["ws"][e], st["K"]).repeat_interleave(_B, dim=0)[:st["N"]]
                torch.matmul(x[a:b], (st["w"][e].float() * s).t(), out=y[a:b])
        return y.to(_TYPES[st["out"]])
    l, E, k = st["l"].float(), st["E"], st["k"]
    live = torch.ones(l.shape[0], device="cuda") if st["mask"] is None else st["mask"].float()
    top = l.amax(-1, keepdim=True)
    e = torch.exp(l - top)
    total = e.sum(-1, keepdim=True)
    p, lse = e / total, (top + torch.log(total)).squeeze(-1)
    if kind == "balance":
        tokens = live.sum()
        counts = torch.zeros(E, dtype=torch.float32, device="cuda")
        counts.index_add_(0, st["ids"].reshape(-1).long(), live.repeat_interleave(k))   # (whole numbers: exact)
        mean_p = (p * live[:, None]).sum(0) / tokens
        losses = torch.stack([E * (counts / (tokens * k) * mean_p).sum(), (lse.square() * live).sum() / tokens])
        return {"losses": losses, "counts": torch.cat([counts, tokens[None]]).to(torch.int32)}
    tokens = st["counts"][E].float()
    f = st["counts"][:E].float() / (tokens * k)
    g = st["dl"][0] * E * p * (f - (p * f).sum(-1, keepdim=True)) + st["dl"][1] * 2.0 * lse[:, None] * p
    return (g * (live / tokens)[:, None]).to(_TYPES[st["out"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------ in 64 bits
def _exact_fp8(v):
    """Scales, and the values over their scales before they are rounded."""
    q, scales = [], []
    for c in range(0, v.shape[1], _B):
        part = v[:, c:c + _B]
        s = part.abs().max(dim=1, keepdim=True).values / 448.0
        scales.append(s.clamp(min=_LEAST))
        q.append(part / scales[-1])
    return torch.cat(q, 1), torch.cat(scales, 1)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        out, h = {}, st["x"].double()
        if st["res"] is not None:
            out["residual"] = (h + st["res"].double()).to(st["res"].dtype).double()
            h = out["residual"]
        norm = torch.sqrt((h * h).sum(1) / case["H"] + st["eps"])
        y = st["w"].double() * (h / norm[:, None])
        if case["out"] != "fp8":
            out["y"] = y
        if case["out"] != "y":
            out["q"], out["scale"] = _exact_fp8(y)
        return out
    if kind == "act":
        v = st["x"].double()
        if case["gated"]:
            g, u = v.split(case["I"], dim=1)
            v = g * torch.sigmoid(g) * u
        q, scale = _exact_fp8(v)
        if case["gated"]:
            scale = scale * st["weights"].double()[st["order"].long()][:, None]
        return {"q": q, "scale": scale}
    if kind == "mm":
        off = st["offsets"].tolist()
        y = torch.empty((off[-1], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            rows = torch.arange(off[e], off[e + 1], device="cuda")
            src = st["order"][rows].long() // case["k"] if case["gather"] else rows
            part = torch.zeros((rows.numel(), case["N"]), dtype=torch.float64, device="cuda")
            for b in range(st["xs"].shape[1]):
                cols = slice(b * _B, (b + 1) * _B)
                dot = st["x"][src][:, cols].double() @ st["w"][e][:, cols].double().t()
                by_row = st["ws"][e, :, b].double().repeat_interleave(_B)[:case["N"]]
                part += dot * st["xs"][src, b].double()[:, None] * by_row
            y[off[e]:off[e + 1]] = part
        return y
    T, k, E = case["T"], case["k"], case["E"]
    rows = torch.arange(T, device="cuda") if st["mask"] is None else st["mask"].nonzero().flatten()
    l = st["l"].double()[rows]
    lse = torch.logsumexp(l, dim=1)
    p = torch.exp(l - lse[:, None])
    M = rows.numel()
    if kind == "balance":
        c = torch.stack([(st["ids"][rows] == e).sum() for e in range(E)])
        losses = torch.stack([E * (c.double() * p.mean(0)).sum() / (M * k), (lse ** 2).mean()])
        return {"losses": losses, "counts": torch.cat([c, torch.tensor([M], device="cuda")]).to(torch.int32)}
    f = st["counts"][:E].double() / (M * k)
    ga, gz = st["dl"].double()
    dl = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    dl[rows] = p * (ga * E / M * (f[None] - (p @ f)[:, None]) + (2.0 * gz / M * lse)[:, None])
    return dl


def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "none": 0}
    if kind == "norm":
        n, b = case["T"] * case["H"], size[case["dtype"]]
        out = (b if case["out"] != "fp8" else 0) + (1 + 4 / _B if case["out"] != "y" else 0)
        return {"bytes": int(n * (b + 2 * size[case["residual"]] + out)) + b * case["H"], "flops": 5 * n}
    if kind == "act":
        n = case["rows"] * case["I"]
        return {"bytes": int(n * (size[case["dtype"]] * (2 if case["gated"] else 1) + 1 + 4 / _B)), "flops": 8 * n}
    T, k, E = case["T"], case["k"], case["E"]
    if kind == "mm":
        N, K, rows = case["N"], case["K"], T * k
        share = [(i + 1) ** -1.1 if case["zipf"] else 1.0 for i in range(E)]
        active = sum(1.0 - (1.0 - min(1.0, k * p / sum(share))) ** T for p in share)   # experts with rows, expected
        return {"bytes": int((T if case["gather"] else rows) * K * (1 + 4 / _B) + active * N * K) + size[case["out"]] * rows * N,
                "flops": 2 * rows * N * K}
    if kind == "balance":
        return {"bytes": T * E * size[case["dtype"]] + 4 * T * k + (T if case["padded"] else 0), "flops": 5 * T * E}
    return {"bytes": T * E * (size[case["dtype"]] + size[case["out"]]) + (T if case["padded"] else 0), "flops": 10 * T * E}
