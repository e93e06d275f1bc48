"""Workloads of the cache-serving operators: rotary positions, attention over a prefix that a batch
shares, the attention weight that cached positions collect, and the eviction that goes by it.

Each case is one call as a serving (or, for the rotary gradient, a training) program makes it. With
`own` false `run` computes it in elementary torch operations; with `own` true through the package.
"""
import math

import torch

own = False

HEADS, LATENT, QK = 128, 512, 576
SCALE = 192 ** -0.5 * (1.0 + 0.1 * math.log(40.0)) ** 2
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the rotary quarter of a decode step's 192-wide query heads, a batch of 64
        {"name": "rope_q_decode", "op": "rope", "rows": 64, "heads": 128, "dim": 192, "offset": 128, "pairs": 32,
         "layout": "interleaved", "dtype": "bf16", "factor": 40.0, "inverse": False, "max_pos": 16384,
         "row_dim": 192 * 128},
        # the rotary key of a prefill chunk, read in place from the 576-wide latent projection
        {"name": "rope_k_chunk", "op": "rope", "rows": 16384, "heads": 1, "dim": 64, "offset": 0, "pairs": 32,
         "layout": "interleaved", "dtype": "bf16", "factor": 40.0, "inverse": False, "max_pos": 1000000,
         "row_dim": 576},
        # the gradient through the indexer's half-layout rotary of 4096 training tokens, in fp32
        {"name": "rope_grad", "op": "rope", "rows": 4096, "heads": 64, "dim": 128, "offset": 0, "pairs": 32,
         "layout": "half", "dtype": "fp32", "factor": 1.0, "inverse": True, "max_pos": 4096, "row_dim": 8192},
        # eight conversations behind one system prompt, a decode step
        {"name": "shared_b8", "op": "shared", "B": 8, "T": 1, "P": 1031, "S": 256},
        # a batch of 64 behind a long shared document, a decode step
        {"name": "shared_b64", "op": "shared", "B": 64, "T": 1, "P": 8192, "S": 512},
        # four sequences that each add a chunk of 128 tokens behind 16384 shared ones
        {"name": "shared_chunk", "op": "shared", "B": 4, "T": 128, "P": 16384, "S": 300},
        # what each cached position got in a dense decode step, added to its running total
        {"name": "weights_decode", "op": "weights", "B": 64, "T": 1, "S": 4096, "k": 0},
        # the same for the 2048 positions that sparse attention selected out of 16384
        {"name": "weights_selected", "op": "weights", "B": 64, "T": 1, "S": 16384, "k": 2048},
        # a causal chunk of 250 tokens over a cache of about 4096
        {"name": "weights_chunk", "op": "weights", "B": 1, "T": 250, "S": 4100, "k": 0},
        # a small batch goes back to its budget after a few hundred new tokens
        {"name": "evict_b8", "op": "evict", "B": 8, "S": 2304, "keep": 2048, "recent": 128, "sinks": 4},
        # a batch of 64 halves its caches
        {"name": "evict_b64", "op": "evict", "B": 64, "S": 16384, "keep": 8192, "recent": 512, "sinks": 4},
        # one long sequence cut to a small budget
        {"name": "evict_long", "op": "evict", "B": 1, "S": 131072, "keep": 8191, "recent": 1000, "sinks": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "weights", "evict"])
    if op == "rope":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        dim = rng.choice([64, 128, 192, 256])
        pairs = rng.choice([16, 32, dim // 4, dim // 2])
        offset = rng.choice([0, dim - 2 * pairs])
        heads = rng.choice([1, 2, 8, 16, 64, 128])
        rows = _log(rng, 1, min(65536, 30000000 // (heads * dim)))
        return {"op": op, "rows": rows, "heads": heads, "dim": dim, "offset": offset, "pairs": pairs,
                "layout": rng.choice(["interleaved", "half"]), "dtype": dtype, "factor": rng.choice([1.0, 4.0, 40.0]),
                "inverse": rng.random() < 0.4, "max_pos": _log(rng, 128, 1000000), "row_dim": heads * dim}
    if op == "shared":
        T = rng.choice([1, 1, 1, 2, 3, _log(rng, 4, 128)])
        P = _log(rng, 1, 16384)
        S = max(T, _log(rng, 1, 2048))
        most = max(1, min(128, 512 * 16684 // (T * (P + S))))
        return {"op": op, "B": _log(rng, 1, most), "T": T, "P": P, "S": S}
    if op == "weights":
        if rng.random() < 0.5:
            S = _log(rng, 64, 16384)
            return {"op": op, "B": _log(rng, 1, max(1, min(64, 262144 // S))), "T": 1, "S": S, "k": 0}
        if rng.random() < 0.5:
            S = _log(rng, 2048, 16384)
            return {"op": op, "B": _log(rng, 1, 64), "T": 1, "S": S, "k": _log(rng, 64, 2048)}
        S = _log(rng, 64, 4096)
        return {"op": op, "B": 1, "T": rng.randint(2, min(S, 250)), "S": S, "k": 0}
    S = _log(rng, 256, 16384)
    keep = rng.randint(S // 4, S - 1)
    return {"op": op, "B": _log(rng, 1, max(1, min(64, 1000000 // S))), "S": S, "keep": keep,
            "recent": rng.randint(0, keep // 4), "sinks": rng.choice([0, 4, 16])}


# ------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def ints(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    if case["op"] == "rope":
        rows, heads, dim = case["rows"], case["heads"], case["dim"]
        dt = DTYPES[case["dtype"]]
        wide = normal(rows, case["row_dim"], dtype=dt)
        st["x"] = wide[:, case["row_dim"] - heads * dim:].unflatten(1, (heads, dim))
        st["pos"] = ints(0, case["max_pos"], (rows,))
        st["out"] = torch.empty((rows, heads, dim), dtype=dt, device="cuda")
        if own:
            import sparse_attention_keys_b200 as dsa
            st["freqs"] = dsa.dsa_rope_freqs(case["pairs"], factor=case["factor"], original_len=4096).cuda()
        else:
            st["freqs"] = torch.tensor(_frequencies(case["pairs"], case["factor"]), dtype=torch.float64, device="cuda")
    elif case["op"] == "shared":
        B, T, P, S = case["B"], case["T"], case["P"], case["S"]
        st["q"] = normal(B, T, HEADS, QK)
        st["prefix"] = normal(P, QK)
        st["kv"] = normal(B, S, QK)
        st["kv_len"] = ints(T, S + 1, (B,))
        # a step's queries are the last T positions of each sequence
        st["q_pos"] = (st["kv_len"][:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        st["out"] = torch.empty((B, T, HEADS, LATENT), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((B, T, HEADS), dtype=torch.float32, device="cuda")
        if own:
            import sparse_attention_keys_b200 as dsa
            size = dsa.dsa_mla_shared_workspace_size(B, T, P, S)
            st["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    elif case["op"] == "weights":
        B, T, S, k = case["B"], case["T"], case["S"], case["k"]
        st["q"] = normal(B, T, HEADS, QK)
        st["kv"] = normal(B, S, QK)
        st["kv_len"] = ints(max(T, S // 2), S + 1, (B,))
        st["q_pos"] = (st["kv_len"][:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        st["acc"] = torch.rand((B, S), generator=g, device="cuda") * HEADS
        st["acc_out"] = torch.empty_like(st["acc"])
        if k:
            # the selection: distinct visible positions in ascending order, -1 behind them
            pick = torch.rand((B, T, S), generator=g, device="cuda")
            s = torch.arange(S, device="cuda", dtype=torch.int32)
            pick.masked_fill_(s > st["q_pos"][..., None], -1.0)
            val, idx = pick.topk(k, dim=-1)
            idx = torch.where(val >= 0, idx, S).sort(dim=-1).values
            st["idx"] = torch.where(idx < S, idx, -1).to(torch.int32).contiguous()
            rows = _rows(st["kv"].float(), st["idx"].clamp(min=0))
            z = SCALE * torch.matmul(st["q"].float(), rows.transpose(-1, -2))
            z = z.masked_fill(st["idx"][:, :, None, :] < 0, -math.inf)
        else:
            z = SCALE * torch.matmul(st["q"].float().flatten(1, 2), st["kv"].float().transpose(1, 2)).unflatten(1, (T, HEADS))
            z = z.masked_fill(~_visible(st)[:, :, None, :], -math.inf)
        st["lse"] = torch.logsumexp(z, dim=-1).contiguous()
        width = k if k else S
        st["w"] = torch.empty((B, T, (width + 3) // 4 * 4), dtype=torch.float32, device="cuda")
    else:
        B, S = case["B"], case["S"]
        st["kv"] = normal(B, S, QK)
        st["kv_len"] = ints((case["keep"] + S) // 2, S + 1, (B,))
        # totals as sparse attention leaves them: a few positions collect most of the weight, some none
        st["acc"] = torch.exp(2.0 * torch.randn((B, S), generator=g, device="cuda"))
        st["acc"] *= torch.rand((B, S), generator=g, device="cuda") > 0.2
        order = torch.rand((B, S), generator=g, device="cuda")
        # an earlier eviction left the first rows in no order; the newer ones follow in theirs
        order[:, case["keep"]:] = 2.0 + torch.arange(S - case["keep"], device="cuda")
        st["pos"] = order.argsort(1).argsort(1).to(torch.int32)
        st["acc_out"], st["pos_out"] = torch.empty_like(st["acc"]), torch.empty_like(st["pos"])
        st["len_out"] = torch.empty_like(st["kv_len"])
        st["src"] = torch.empty((B, case["keep"]), dtype=torch.int32, device="cuda")
        if own:
            import sparse_attention_keys_b200 as dsa
            size = dsa.dsa_cache_evict_workspace_size(B, S, case["keep"])
            st["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return st


def _visible(st):
    s = torch.arange(st["kv"].shape[1], device="cuda", dtype=torch.int32)
    return (s <= st["q_pos"][..., None]) & (s < st["kv_len"][:, None, None])


def _rows(kv, idx):
    """kv [B,S,D] at idx [B,T,k] -> [B,T,k,D]"""
    b = torch.arange(kv.shape[0], device=kv.device)[:, None, None]
    return kv[b, idx.long()]


def _frequencies(pairs, factor, theta=10000.0, original=4096, beta_fast=32.0, beta_slow=1.0):
    """Radians per position; for factor > 1 the YaRN blend of kept and slowed frequencies."""
    dim = 2 * pairs

    def turns_at(n):
        return dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta))

    low, high = max(math.floor(turns_at(beta_fast)), 0), min(math.ceil(turns_at(beta_slow)), dim - 1)
    if low == high:
        high += 0.001
    out = []
    for i in range(pairs):
        f = theta ** (-2.0 * i / dim)
        keep = 1.0 - min(max((i - low) / (high - low), 0.0), 1.0)
        out.append(f * keep + f / factor * (1.0 - keep) if factor > 1.0 else f)
    return out


# --------------------------------------------------------------------------------------------- run
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import sparse_attention_keys_b200 as dsa
    case = st["case"]
    if case["op"] == "rope":
        return dsa.dsa_rope(st["x"], st["pos"], st["freqs"], offset=case["offset"],
                            interleaved=case["layout"] == "interleaved", inverse=case["inverse"], out=st["out"])
    if case["op"] == "shared":
        return dsa.dsa_mla_shared(st["q"], st["prefix"], st["kv"], st["q_pos"], st["kv_len"], out=st["out"],
                                  lse=st["lse"], workspace=st["workspace"])
    if case["op"] == "weights":
        if case["k"]:
            w, acc = dsa.dsa_mla_weights_selected(st["q"], st["kv"], st["idx"], st["lse"], acc=st["acc"],
                                                  acc_out=st["acc_out"], w=st["w"])
        else:
            w, acc = dsa.dsa_mla_weights(st["q"], st["kv"], st["lse"], st["q_pos"], st["kv_len"], acc=st["acc"],
                                         acc_out=st["acc_out"], w=st["w"])
        return w[..., :case["k"] or case["S"]], acc
    dsa.dsa_cache_evict(st["acc"], st["pos"], st["kv_len"], case["keep"], recent=case["recent"], sinks=case["sinks"],
                        kv=st["kv"], acc_out=st["acc_out"], pos_out=st["pos_out"], kv_len_out=st["len_out"],
                        src=st["src"], workspace=st["workspace"])
    return _kept(st)


def _kept(st):
    """The evicted cache's live rows: every sequence keeps `keep` (all of them are longer)."""
    keep = st["case"]["keep"]
    return {"kv": st["kv"][:, :keep], "acc": st["acc_out"][:, :keep], "pos": st["pos_out"][:, :keep],
            "kv_len": st["len_out"], "src": st["src"]}


def _run_plain(st):
    case = st["case"]
    if case["op"] == "rope":
        x = st["x"].float()
        angle = st["pos"].double()[:, None] * st["freqs"]
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        if case["inverse"]:
            sin = -sin
        st["out"].copy_(_rotate(x, cos, sin, case))
        return st["out"]
    if case["op"] == "shared":
        B, T = case["B"], case["T"]
        q, prefix, kv = st["q"].float(), st["prefix"].float(), st["kv"].float()
        zp = SCALE * torch.matmul(q, prefix.t())
        zs = SCALE * torch.matmul(q.flatten(1, 2), kv.transpose(1, 2)).unflatten(1, (T, HEADS))
        zs.masked_fill_(~_visible(st)[:, :, None, :], -math.inf)
        m = torch.maximum(zp.amax(-1), zs.amax(-1))
        zp.sub_(m[..., None]).exp_()
        zs.sub_(m[..., None]).exp_()
        total = zp.sum(-1) + zs.sum(-1)
        o = torch.matmul(zp, prefix[:, :LATENT])
        o += torch.matmul(zs.flatten(1, 2), kv[..., :LATENT]).unflatten(1, (T, HEADS))
        st["out"].copy_(o / total[..., None])
        torch.add(m, torch.log(total), out=st["lse"])
        return st["out"], st["lse"]
    if case["op"] == "weights":
        T = case["T"]
        q, kv, lse = st["q"].float(), st["kv"].float(), st["lse"]
        if case["k"]:
            z = SCALE * torch.matmul(q, _rows(kv, st["idx"].clamp(min=0)).transpose(-1, -2))
            w = torch.exp(z - lse[..., None]).sum(2).masked_fill(st["idx"] < 0, 0.0)
            # a row beyond the cache takes the unused slots
            acc = torch.cat([st["acc"], torch.zeros_like(st["acc"][:, :1])], 1)
            to = torch.where(st["idx"] >= 0, st["idx"], case["S"]).long()
            for t in range(T):
                acc.scatter_add_(1, to[:, t], w[:, t])
            st["acc_out"].copy_(acc[:, :case["S"]])
        else:
            z = SCALE * torch.matmul(q.flatten(1, 2), kv.transpose(1, 2)).unflatten(1, (T, HEADS))
            w = torch.exp(z - lse[..., None]).sum(2).masked_fill(~_visible(st), 0.0)
            torch.add(st["acc"], w.sum(1), out=st["acc_out"])
        return w, st["acc_out"]
    # evict: the protected rows, then the heaviest, ties to the lower row; kept rows that lie behind
    # the budget move, in their order, into the rows that were given up before it
    keep, n = case["keep"], st["kv_len"].long()
    B, S = st["acc"].shape
    row = torch.arange(S, device="cuda")
    live = row < n[:, None]
    newest = st["pos"].masked_fill(~live, -1).amax(1, keepdim=True)
    safe = (st["pos"] > newest - case["recent"]) | (st["pos"] < case["sinks"])
    order = torch.argsort(st["acc"], dim=1, descending=True, stable=True)
    klass = torch.where(live, torch.where(safe, 0, 1), 2)
    order = order.gather(1, torch.argsort(klass.gather(1, order), dim=1, stable=True))
    kept = torch.zeros_like(live).scatter_(1, order[:, :keep], True)
    src = row[:keep].expand(B, keep).clone()
    stays = kept[:, :keep]
    # the i-th hole takes the i-th mover
    movers = kept & (row >= keep)
    nth = torch.argsort((~movers).to(torch.int8), dim=1, stable=True)
    hole = torch.cumsum((~stays).long(), 1) - 1
    src = torch.where(stays, src, nth.gather(1, hole.clamp(min=0)))
    b = torch.arange(B, device="cuda")[:, None]
    st["kv"][:, :keep] = st["kv"][b, src]
    st["acc_out"][:, :keep] = st["acc"].gather(1, src)
    st["pos_out"][:, :keep] = st["pos"].gather(1, src)
    st["len_out"].copy_(n.clamp(max=keep))
    st["src"].copy_(src)
    return _kept(st)


def _rotate(x, cos, sin, case):
    lo, pairs = case["offset"], case["pairs"]
    y = x.clone()
    if case["layout"] == "interleaved":
        first, second = slice(lo, lo + 2 * pairs, 2), slice(lo + 1, lo + 2 * pairs, 2)
    else:
        first, second = slice(lo, lo + pairs), slice(lo + pairs, lo + 2 * pairs)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = a * sin + b * cos
    return y


# ------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        x = st["x"].double()
        lo, n = case["offset"], case["pairs"]
        f = torch.tensor(_frequencies(n, case["factor"]), dtype=torch.float64, device="cuda")
        # a pair is a complex number; position p turns it by p * f
        turn = torch.polar(torch.ones_like(f), f * (-1.0 if case["inverse"] else 1.0) * st["pos"].double()[:, None])
        rot = x[..., lo:lo + 2 * n]
        if case["layout"] == "half":
            z = torch.complex(rot[..., :n].contiguous(), rot[..., n:].contiguous()) * turn[:, None]
            rot = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(rot.unflatten(-1, (n, 2)).contiguous()) * turn[:, None]
            rot = torch.view_as_real(z).flatten(-2)
        return torch.cat([x[..., :lo], rot, x[..., lo + 2 * n:]], -1)
    if case["op"] == "shared":
        B, T = case["B"], case["T"]
        if B * T * HEADS * (case["P"] + case["S"]) * 2 * (QK + LATENT) > 4e12:
            return None
        out = torch.empty((B, T, HEADS, LATENT), dtype=torch.float64, device="cuda")
        lse = torch.empty((B, T, HEADS), dtype=torch.float64, device="cuda")
        prefix = st["prefix"].double()
        for b in range(B):
            for t in range(T):
                seen = min(int(st["q_pos"][b, t]) + 1, int(st["kv_len"][b]))
                keys = torch.cat([prefix, st["kv"][b, :seen].double()])
                z = (st["q"][b, t].double() @ keys.t()) * SCALE
                lse[b, t] = torch.logsumexp(z, -1)
                out[b, t] = torch.softmax(z, -1) @ keys[:, :LATENT]
        return out, lse
    if case["op"] == "weights":
        B, T, S, k = case["B"], case["T"], case["S"], case["k"]
        w = torch.zeros((B, T, k or S), dtype=torch.float64, device="cuda")
        acc = st["acc"].double()
        for b in range(B):
            kv = st["kv"][b].double()
            for t in range(T):
                if k:
                    at = st["idx"][b, t]
                    at = at[at >= 0].long()
                else:
                    at = torch.arange(min(int(st["q_pos"][b, t]) + 1, int(st["kv_len"][b])), device="cuda")
                z = SCALE * (st["q"][b, t].double() @ kv[at].t())
                p = torch.exp(z - st["lse"][b, t].double()[:, None]).sum(0)
                w[b, t, :len(at)] = p
                acc[b, at] += p
        return w, acc
    # evict: whole numbers and copies, from the definition one sequence at a time on the host
    keep = case["keep"]
    B = case["B"]
    src = torch.empty((B, keep), dtype=torch.int64)
    acc, pos, lens = st["acc"].cpu(), st["pos"].cpu(), st["kv_len"].cpu()
    for b in range(B):
        n = int(lens[b])
        a, p = acc[b, :n].tolist(), pos[b, :n].tolist()
        newest = max(p)
        safe = [p[r] > newest - case["recent"] or p[r] < case["sinks"] for r in range(n)]
        ranked = sorted(range(n), key=lambda r: (not safe[r], -a[r], r))
        kept = sorted(ranked[:keep])
        inside = [r for r in kept if r < keep]
        movers = iter([r for r in kept if r >= keep])
        there = set(inside)
        src[b] = torch.tensor([i if i in there else next(movers) for i in range(keep)])
    at = src.cuda()
    b = torch.arange(B, device="cuda")[:, None]
    return {"kv": st["kv"][b, at].double(), "acc": st["acc"].gather(1, at).double(),
            "pos": st["pos"].gather(1, at), "kv_len": st["kv_len"].clamp(max=keep), "src": at.to(torch.int32)}


# -------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["rows"] + 8 * case["pairs"],
                "flops": 6 * n * case["pairs"]}
    if case["op"] == "shared":
        B, T, P = case["B"], case["T"], case["P"]
        # lengths are uniform on [T, S]; a query sees half a chunk less than its sequence, on average
        own_rows = (T + case["S"]) / 2
        seen = P + own_rows - (T - 1) / 2
        return {"bytes": int(B * T * HEADS * (2 * QK + 2 * LATENT + 4) + 2 * QK * (P + B * own_rows) + 4 * B * (T + 1)),
                "flops": int(B * T * HEADS * seen * 2 * (QK + LATENT))}
    if case["op"] == "weights":
        B, T, S, k = case["B"], case["T"], case["S"], case["k"]
        rows = (max(T, S // 2) + S) / 2
        if k:
            touched = min(k, rows)
            return {"bytes": int(B * T * (HEADS * (2 * QK + 4) + touched * 2 * QK + 8 * k) + 8 * B * S),
                    "flops": int(B * T * HEADS * touched * 2 * QK)}
        seen = rows - (T - 1) / 2
        return {"bytes": int(B * T * (HEADS * (2 * QK + 4) + 4 * S) + B * (rows * 2 * QK + 8 * S)),
                "flops": int(B * T * HEADS * seen * 2 * QK)}
    B, S, keep = case["B"], case["S"], case["keep"]
    n = ((keep + S) // 2 + S) / 2
    # the recent rows that lie behind the budget move, and of the others their share of the rest
    new = n - keep
    recent = min(case["recent"], new)
    moved = recent + (new - recent) * (keep - recent) / max(n - recent, 1)
    return {"bytes": int(B * (n * 8 + keep * 12 + moved * 4 * QK)), "flops": int(B * n * 4)}
