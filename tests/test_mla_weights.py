"""dsa_mla_weights and dsa_mla_weights_selected: head-summed attention weights against the formula in 64
bits, and the whole loop they belong to.

Tolerance. A score is off by d = 576 * 2^-24 * scale * sum |q k| (fp32 accumulation of exact products),
its base-2 exponent by two roundings of 2^-24 of |z| and |lse| (each times log2 e in fp32), the approximate
exponential by 2^-21, the sum over 128 heads by 2^-17: |dw| <= sum_h p (d + 2^-22 (|z| + |lse|) + 2^-16)
(p grows with e^d: 2 d is taken). A sum over T queries adds T 2^-24 of itself."""
import ctypes

import pytest
import torch

import __graft_entry__

__graft_entry__._build_module().build()
import sparse_attention_keys_b200 as dsa  # noqa: E402

gpu = pytest.mark.gpu
SCALE = dsa.MLA_SOFTMAX_SCALE


def test_abi_refusals():
    p, odd, n = ctypes.c_void_p(64), ctypes.c_void_p(65), None
    f = ctypes.c_float
    #        q kv lse q_pos kv_len B T S scale w ld acc acc_out stream
    dense = [p, p, p, p, p, 2, 1, 64, f(0.1), p, 64, p, p, n]
    #        q kv idx lse B T S k scale w ld acc acc_out stream
    picked = [p, p, p, p, 2, 1, 64, 16, f(0.1), p, 16, p, p, n]

    def bad(call, good, **kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return call(*a)

    def d(**kw):
        return bad(dsa.lib.dsa_mla_weights, dense, **kw)

    def s(**kw):
        return bad(dsa.lib.dsa_mla_weights_selected, picked, **kw)

    assert d(_5=0) == 1 and d(_5=65536) == 1 and d(_6=0) == 1 and d(_7=0) == 1 and d(_7=(1 << 20) + 1) == 1
    assert d(_10=63) == 1 and d(_10=60) == 1 and d(_10=66) == 1 and d(_8=f(0.0)) == 1 and d(_8=f(float("inf"))) == 1
    assert d(_11=n) == 1 and d(_12=n) == 1                          # a sum needs both
    for i in (0, 1, 2, 3, 4, 9):
        assert d(**{f"_{i}": n}) == 1 and d(**{f"_{i}": odd}) == 1
    for i in (0, 1, 2, 3, 9):
        assert s(**{f"_{i}": n}) == 1 and s(**{f"_{i}": odd}) == 1
    assert s(_4=0) == 1 and s(_5=0) == 1 and s(_6=0) == 1 and s(_7=0) == 1 and s(_10=12) == 1 and s(_10=18) == 1
    assert s(_5=1 << 23) == 1 and s(_11=odd) == 1 and s(_12=odd) == 1


def test_binding_refusals():
    q = torch.zeros(1, 1, 128, 576, dtype=torch.bfloat16)
    lse = torch.zeros(1, 1, 128)
    with pytest.raises(ValueError):                                 # host memory
        dsa.dsa_mla_weights(q, q[0], lse, None, None)
    with pytest.raises(TypeError):
        dsa.dsa_mla_weights_selected(q, q[0], torch.zeros(1, 1, 4), lse)


# ------------------------------------------------------------------------------------------- GPU
def make(B, T, S, seed=0, lens=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((B, T, 128, 576), generator=g, device="cuda").bfloat16()
    kv = torch.randn((B, S, 576), generator=g, device="cuda").bfloat16()
    if lens is None:
        lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda")
    kv_len = torch.as_tensor(lens, dtype=torch.int32, device="cuda")
    q_pos = (kv_len[:, None] - T + torch.arange(T, device="cuda")).to(torch.int32)
    return q, kv, q_pos, kv_len


def reference(q, kv, lse, rows):
    """rows: [B][T] lists of row indices -> ([B][T] weights, [B][T] tolerances) in float64"""
    out = []
    for b in range(q.shape[0]):
        line = []
        for t in range(q.shape[1]):
            k = kv[b, rows[b][t]].double()
            x = q[b, t].double()
            z = SCALE * x @ k.t()
            ls = lse[b, t].double()[:, None]
            p = torch.exp(z - ls)
            d = 576 * 2.0 ** -24 * SCALE * (x.abs() @ k.abs().t())
            line.append((p.sum(0), (p * (2 * d + 2.0 ** -22 * (z.abs() + ls.abs()) + 2.0 ** -16)).sum(0)))
        out.append(line)
    return out


def visible(q_pos, kv_len, S, b, t):
    return max(0, min(int(q_pos[b, t]) + 1, int(kv_len[b]), S))


def lse_of(q, kv, rows):
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    for b in range(q.shape[0]):
        for t in range(q.shape[1]):
            lse[b, t] = torch.logsumexp(SCALE * q[b, t].double() @ kv[b, rows[b][t]].double().t(), -1)
    return lse.float()


def close(got, want, tol):
    assert bool(((got.double() - want).abs() <= tol).all()), float(((got.double() - want).abs() - tol).max())


@gpu
@pytest.mark.parametrize("B,T,S", [(1, 1, 1), (2, 1, 127), (3, 1, 130), (5, 1, 1031), (1, 2, 5), (2, 3, 260), (1, 7, 128),
                                   (200, 1, 40), (3, 40, 300)])
def test_weights(B, T, S):
    q, kv, q_pos, kv_len = make(B, T, S, seed=S)
    rows = [[torch.arange(visible(q_pos, kv_len, S, b, t), device="cuda") for t in range(T)] for b in range(B)]
    lse = lse_of(q, kv, rows)
    acc = torch.rand((B, S), device="cuda")
    ld = (S + 3) // 4 * 4 + 4
    w = torch.full((B, T, ld), -3.0, device="cuda")
    out = torch.empty_like(acc)
    dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len, acc=acc, acc_out=out, w=w)
    assert dsa.dsa_get_device_status() == 0
    ref = reference(q, kv, lse, rows)
    assert bool((w[..., S:] == -3.0).all())
    for b in range(B):
        total, slack = acc[b].double(), torch.zeros(S, dtype=torch.float64, device="cuda")
        for t in range(T):
            n = len(rows[b][t])
            close(w[b, t, :n], *ref[b][t])
            assert bool((w[b, t, n:S] == 0).all())
            total[:n] += ref[b][t][0]
            slack[:n] += ref[b][t][1]
        close(out[b], total, slack + (T + 1) * 2.0 ** -24 * total)
        assert T > 1 or abs(float(w[b, 0, :S].sum()) - (128 if len(rows[b][0]) else 0)) < 1e-2
    # without a sum, and in place: the same bits
    w2, none = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    assert none is None and torch.equal(w2[..., :S], w[..., :S])
    dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len, acc=acc, w=w)
    assert torch.equal(acc, out)


@gpu
def test_a_new_query_every_tile():
    """Many queries in a row for each pair of CTAs, one tile each, whose lse lie far apart."""
    B, T, S = 2, 800, 60
    q, kv, q_pos, kv_len = make(B, T, S, seed=9, lens=[S, S - 1])
    q *= (0.25 * (1 + torch.arange(T, device="cuda") % 7)).to(q.dtype)[None, :, None, None]
    q_pos.fill_(S)
    rows = [[torch.arange(visible(q_pos, kv_len, S, b, t), device="cuda") for t in range(T)] for b in range(B)]
    lse = lse_of(q, kv, rows)
    w, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    idx = torch.arange(S, device="cuda", dtype=torch.int32).expand(B, T, S).contiguous()
    idx[1, :, S - 1] = -1
    ws, _ = dsa.dsa_mla_weights_selected(q, kv, idx, lse)
    assert dsa.dsa_get_device_status() == 0
    ref = reference(q, kv, lse, rows)
    for b in range(B):
        n = len(rows[b][0])
        want, tol = (torch.stack([r[i] for r in ref[b]]) for i in (0, 1))
        for got in (w, ws):
            close(got[b, :, :n], want, tol)
            assert bool((got[b, :, n:S] == 0).all())


@gpu
def test_hidden_rows_lengths_and_minus_infinity():
    lens = [0, 1, 128, 129, 256, 300, 77]
    q, kv, q_pos, kv_len = make(7, 2, 256, seed=2, lens=lens)
    q_pos[4] = torch.tensor([-5, 1 << 30])
    rows = [[torch.arange(visible(q_pos, kv_len, 256, b, t), device="cuda") for t in range(2)] for b in range(7)]
    lse = lse_of(q, kv, rows)                                      # -inf where nothing is seen
    assert bool(lse[0].isinf().all())
    clean, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    for b in range(7):
        kv[b, len(rows[b][1]):] = float("nan")
    got, acc = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len, acc=torch.zeros((7, 256), device="cuda"))
    assert torch.equal(clean, got) and bool(acc.isfinite().all()) and torch.equal(acc, got.sum(1))
    ref = reference(q, kv, lse, rows)
    for b in range(7):
        for t in range(2):
            close(got[b, t, :len(rows[b][t])], *ref[b][t])
            assert bool((got[b, t, len(rows[b][t]):] == 0).all())


@gpu
@pytest.mark.parametrize("B,T,S,k", [(1, 1, 1, 1), (3, 1, 700, 130), (2, 4, 300, 50), (1, 1, 20000, 2048), (70, 2, 90, 7),
                                     (1, 60, 9000, 256)])
def test_selected(B, T, S, k):
    q, kv, _, _ = make(B, T, S, seed=k)
    g = torch.Generator(device="cuda").manual_seed(k)
    idx = torch.rand((B, T, S), generator=g, device="cuda").topk(min(k, S), -1).indices
    idx = torch.nn.functional.pad(idx, (0, k - min(k, S)), value=-1).to(torch.int32)
    holes = torch.rand((B, T, k), generator=g, device="cuda") < 0.2             # unused slots anywhere
    holes[..., 0] = False
    idx = torch.where(holes, -1, idx).contiguous()
    rows = [[idx[b, t][idx[b, t] >= 0].long() for t in range(T)] for b in range(B)]
    lse = lse_of(q, kv, rows)
    acc = torch.rand((B, S), device="cuda")
    w, out = dsa.dsa_mla_weights_selected(q, kv, idx, lse, acc=acc, acc_out=torch.empty_like(acc))
    assert dsa.dsa_get_device_status() == 0
    ref = reference(q, kv, lse, rows)
    for b in range(B):
        total, slack = acc[b].double(), torch.zeros(S, dtype=torch.float64, device="cuda")
        for t in range(T):
            close(w[b, t, :k][idx[b, t] >= 0], *ref[b][t])
            assert bool((w[b, t, :k][idx[b, t] < 0] == 0).all())
            total[rows[b][t]] += ref[b][t][0]
            slack[rows[b][t]] += ref[b][t][1]
        close(out[b], total, slack + (T + 1) * 2.0 ** -24 * total)
    w2, _ = dsa.dsa_mla_weights_selected(q, kv, idx, lse, acc=acc)
    assert torch.equal(acc, out) and torch.equal(w2[..., :k], w[..., :k])


@gpu
def test_selected_index_past_the_cache():
    """It is recorded and counts as unused; NaN in rows that nobody selected stays there."""
    q, kv, _, _ = make(1, 1, 64, seed=5)
    idx = torch.arange(10, device="cuda", dtype=torch.int32)[None, None].contiguous()
    kv[0, 10:] = float("nan")
    lse = lse_of(q, kv, [[torch.arange(10, device="cuda")]])
    want, a = dsa.dsa_mla_weights_selected(q, kv, idx, lse, acc=torch.zeros((1, 64), device="cuda"))
    assert dsa.dsa_get_device_status() == 0 and bool((a[0, 10:] == 0).all())
    idx2 = torch.cat([idx, torch.full((1, 1, 2), 64, dtype=torch.int32, device="cuda")], -1)
    got, a2 = dsa.dsa_mla_weights_selected(q, kv, idx2, lse, acc=torch.zeros((1, 64), device="cuda"))
    assert dsa.dsa_get_device_status() == 5
    assert torch.equal(got[..., :10], want[..., :10]) and bool((got[..., 10:] == 0).all()) and torch.equal(a, a2)


@gpu
def test_streams_graphs_and_refusals():
    q, kv, q_pos, kv_len = make(4, 1, 400, seed=6, lens=[400, 0, 130, 7])
    out, lse = dsa.dsa_mla_shared(q, None, kv, q_pos, kv_len)
    want, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len, stream=side)
    b, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    acc, w = torch.zeros((4, 400), device="cuda"), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len, acc=acc, w=w)
    for i in range(1, 4):
        g.replay()
        assert torch.equal(w, want)
    assert bool((acc - 3 * want[:, 0]).abs().max() <= 3 * 2.0 ** -23 * acc.max())
    good = dict(q=q, kv=kv, lse=lse, q_pos=q_pos, kv_len=kv_len)
    for bad in (dict(q=q[:3]), dict(kv=kv[..., :512].contiguous()), dict(lse=lse[..., :64].contiguous()), dict(q_pos=q_pos[:3]),
                dict(kv_len=kv_len.long()), dict(acc_out=acc), dict(acc=acc[:, :399].contiguous()), dict(w=w[..., :396].contiguous()),
                dict(w=torch.empty((4, 1, 402), device="cuda")), dict(lse=lse.cpu())):
        with pytest.raises((ValueError, TypeError)):
            dsa.dsa_mla_weights(**{**good, **bad})


@gpu
def test_cache_past_32_bit_offsets():
    B, S = 4, 940000
    kv = torch.zeros((B, S, 576), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(3)
    kv[3, -300:] = torch.randn((300, 576), generator=g, device="cuda").bfloat16()
    q = torch.randn((B, 1, 128, 576), generator=g, device="cuda").bfloat16()
    idx = (S - 300 + torch.randperm(300, device="cuda", generator=g)).to(torch.int32).expand(B, 1, 300).contiguous()
    lse = torch.full((B, 1, 128), 9.0, device="cuda")
    w, _ = dsa.dsa_mla_weights_selected(q, kv, idx, lse)
    close(w[3, 0], *reference(q[3:], kv[3:], lse[3:], [[idx[3, 0].long()]])[0][0])


@gpu
def test_the_whole_loop():
    """As a server runs it: two sequences behind one prompt decode with a budget of 40 own rows. The rotary key
    enters the cache, attention runs over prompt and own rows, its lse gives the weights, and every eighth step
    evicts. Checked against the same loop in float64 that follows the kernel's choice of rows."""
    B, P, S, keep, steps = 2, 150, 48, 40, 30
    g = torch.Generator(device="cuda").manual_seed(11)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda").bfloat16()

    prefix, kv = normal(P, 576), torch.full((B, S, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    k8 = torch.zeros((B, S, 128), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((B, S), device="cuda")
    pos = torch.zeros((B, S), dtype=torch.int32, device="cuda")
    acc = torch.zeros((B, S), device="cuda")
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    freqs = dsa.dsa_rope_freqs(32, factor=40.0, original_len=4096).cuda()
    held = [dict() for _ in range(B)]                                # position -> (row of the cache, weight)
    for step in range(steps):
        n = int(kv_len[0])
        latent = normal(B, 576)
        at = torch.full((B,), P + step, dtype=torch.int32, device="cuda")
        kv[:, n] = dsa.dsa_rope(latent, at, freqs, offset=512, interleaved=True)
        k8[:, n], ks[:, n], pos[:, n], acc[:, n] = step, float(step), step, 0.0
        kv_len += 1
        for b in range(B):
            held[b][step] = [kv[b, n].double(), torch.zeros((), dtype=torch.float64, device="cuda")]
        q = normal(B, 1, 128, 576)
        q_pos = (kv_len[:, None] - 1).contiguous()
        out, lse = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
        w, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len, acc=acc)
        for b in range(B):
            rows = torch.stack([r for r, _ in held[b].values()])
            keys = torch.cat([prefix.double(), rows])
            p = torch.softmax(SCALE * q[b, 0].double() @ keys.t(), -1)
            want = p @ keys[:, :512]
            # bf16 weights and output: 2^-8 each, with room for the scores' 2^-9
            assert bool(((out[b, 0].double() - want).abs() <= 2.0 ** -6 * (p @ keys[:, :512].abs())).all())
            for h, x in zip(held[b].values(), p[:, P:].sum(0)):
                h[1] += x
        if int(kv_len[0]) == S:
            dsa.dsa_cache_evict(acc, pos, kv_len, keep, recent=8, sinks=2, kv=kv, k8=k8, k_scale=ks)
            for b in range(B):
                alive = pos[b, :keep].tolist()
                ranked = sorted(held[b], key=lambda s: (not (s > step - 8 or s < 2), -float(held[b][s][1])))
                # the choice agrees up to weights that fp32 cannot tell apart
                border = float(held[b][ranked[keep - 1]][1])
                for s in set(alive) ^ set(ranked[:keep]):
                    assert abs(float(held[b][s][1]) - border) <= 1e-4 * border
                held[b] = {s: held[b][s] for s in alive}
        for b in range(B):
            m = int(kv_len[b])
            order = pos[b, :m].tolist()
            assert sorted(order) == sorted(held[b]) and k8[b, :m, 0].tolist() == order and ks[b, :m].tolist() == order
            assert torch.equal(kv[b, :m].double(), torch.stack([held[b][s][0] for s in order]))
            ref = torch.stack([held[b][s][1] for s in order])
            assert bool(((acc[b, :m].double() - ref).abs() <= 1e-3 * ref + 1e-6).all())
    assert dsa.dsa_get_device_status() == 0


@gpu
def test_prefix_and_own_rows_with_the_lse_of_both():
    """A prefix that the batch shares is one sequence with every query; with the lse over prefix and own rows the two
    calls' weights are those of one softmax."""
    B, T, P, S = 3, 2, 150, 70
    q, kv, q_pos, kv_len = make(B, T, S, seed=4, lens=[S, 0, 33])
    prefix = make(1, 1, P, seed=5)[1]
    _, lse = dsa.dsa_mla_shared(q, prefix[0], kv, q_pos, kv_len)
    own, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    everywhere = torch.full((1, B * T), P - 1, dtype=torch.int32, device="cuda")
    before = torch.rand((1, P), device="cuda")
    shared, acc = dsa.dsa_mla_weights(q.view(1, B * T, 128, 576), prefix, lse.view(1, B * T, 128), everywhere,
                                      torch.tensor([P], dtype=torch.int32, device="cuda"), acc=before.clone())
    assert dsa.dsa_get_device_status() == 0
    rows = [[torch.arange(visible(q_pos, kv_len, S, b, t), device="cuda") for t in range(T)] for b in range(B)]
    ref = reference(q, kv, lse, rows)
    total, slack = before[0].double(), torch.zeros(P, dtype=torch.float64, device="cuda")
    every = [[torch.arange(P, device="cuda")]]
    for b in range(B):
        for t in range(T):
            i = b * T + t
            want, tol = reference(q[b:b + 1, t:t + 1], prefix, lse[b:b + 1, t:t + 1], every)[0][0]
            close(shared[0, i, :P], want, tol)
            close(own[b, t, :len(rows[b][t])], *ref[b][t])
            # one softmax over both, 128 heads of it; its lse is off by the scores' error d (within 2 d of the tolerance)
            both, room = want.sum() + ref[b][t][0].sum(), tol.sum() + ref[b][t][1].sum()
            assert abs(float(both) - 128) <= 2 * float(room)
            total += want
            slack += tol
    close(acc[0], total, slack + (B * T + 1) * 2.0 ** -24 * total)


@gpu
def test_the_sparse_loop():
    """As the path decodes: the indexer's keys enter their cache, dsa_index_topk selects, dsa_sparse_mla attends, its lse
    gives the selected rows' weights, and a full cache is evicted with the indexer's codes and scales. The rows' order
    changes nothing: the same selection, as positions, as from a cache in the order of positions, and the attention is
    that of the selected rows in 64 bits."""
    B, S, keep, k, start, steps = 3, 96, 64, 24, 80, 60
    g = torch.Generator(device="cuda").manual_seed(17)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda")

    table = dsa.dsa_rope_table(1024).cuda()
    k8, ks = torch.zeros((B, S, 128), dtype=torch.uint8, device="cuda"), torch.zeros((B, S), device="cuda")
    kv = torch.zeros((B, S, 576), dtype=torch.bfloat16, device="cuda")
    pos, acc = torch.zeros((B, S), dtype=torch.int32, device="cuda"), torch.zeros((B, S), device="cuda")
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    first = torch.arange(B, device="cuda") * S
    # every key at its position, never moved: what the evicted cache is compared with
    n_all = start + steps
    all8, all_s = torch.zeros((B, n_all, 128), dtype=torch.uint8, device="cuda"), torch.zeros((B, n_all), device="cuda")
    all_kv = torch.zeros((B, n_all, 576), dtype=torch.bfloat16, device="cuda")
    evictions = 0

    def append(at):
        """One token per sequence, at position `at`."""
        n = int(kv_len[0])
        p = torch.full((B,), at, dtype=torch.int32, device="cuda")
        key, row = normal(B, 128), normal(B, 576).bfloat16()
        dsa.dsa_index_keys(key, p, table, out_fp8=k8, out_scale=ks, dst_row=first + n)
        dsa.dsa_index_keys(key, p, table, out_fp8=all8, out_scale=all_s, dst_row=torch.arange(B, device="cuda") * n_all + at)
        kv[:, n], all_kv[:, at], pos[:, n], acc[:, n] = row, row, at, 0.0
        kv_len.add_(1)

    for at in range(start):
        append(at)
    for step in range(steps):
        at = start + step
        append(at)
        n = int(kv_len[0])
        p = torch.full((B,), at, dtype=torch.int32, device="cuda")
        q8, qs = dsa.dsa_index_keys(normal(B, 64, 128), p, table)
        q8, qs, w = q8[:, None].contiguous(), qs[:, None].contiguous(), normal(B, 1, 64)
        q_pos = (kv_len[:, None] - 1).contiguous()
        idx = dsa.dsa_index_topk(q8, qs, w, k8, ks, q_pos, kv_len, k)
        picked = pos.gather(1, idx[:, 0].long()).sort(1).values
        # the same rows in the order of their positions
        order = pos[:, :n].sort(1).values.long()
        bi = torch.arange(B, device="cuda")[:, None]
        sorted8, sorted_s = all8[bi, order].contiguous(), all_s[bi, order].contiguous()
        ref = dsa.dsa_index_topk(q8, qs, w, sorted8, sorted_s, q_pos, kv_len, k)
        assert torch.equal(picked.long(), order.gather(1, ref[:, 0].long()).sort(1).values)
        q = normal(B, 1, 128, 576).bfloat16()
        out, lse = dsa.dsa_sparse_mla(q, kv, idx)
        before = acc.clone()
        weights, _ = dsa.dsa_mla_weights_selected(q, kv, idx, lse, acc=acc)
        rows = [[idx[b, 0].long()] for b in range(B)]
        ref_w = reference(q, kv, lse, rows)
        for b in range(B):
            keys = all_kv[b, pos[b, idx[b, 0].long()].long()].double()
            pr = torch.softmax(SCALE * q[b, 0].double() @ keys.t(), -1)
            # bf16 weights and output: 2^-8 each, with room for the scores' 2^-9
            assert bool(((out[b, 0].double() - pr @ keys[:, :512]).abs() <= 2.0 ** -6 * (pr @ keys[:, :512].abs())).all())
            close(weights[b, 0, :k], *ref_w[b][0])
            want = before[b].double().index_add(0, rows[b][0], ref_w[b][0][0])
            room = torch.zeros_like(want).index_add(0, rows[b][0], ref_w[b][0][1])
            close(acc[b], want, room + 2.0 ** -23 * want)
        if n == S:
            held = [dict(zip(pos[b].tolist(), acc[b].tolist())) for b in range(B)]
            dsa.dsa_cache_evict(acc, pos, kv_len, keep, recent=8, sinks=2, kv=kv, k8=k8, k_scale=ks)
            evictions += 1
            assert kv_len.tolist() == [keep] * B
            for b in range(B):
                at_row = pos[b, :keep].long()
                ranked = sorted(held[b], key=lambda s: (not (s > at - 8 or s < 2), -held[b][s]))
                cut = held[b][ranked[keep - 1]]
                for s in set(at_row.tolist()) ^ set(ranked[:keep]):  # positions of equal weight may stand for one another
                    assert held[b][s] == cut
                assert torch.equal(k8[b, :keep], all8[b, at_row]) and torch.equal(ks[b, :keep], all_s[b, at_row])
                assert torch.equal(kv[b, :keep], all_kv[b, at_row])
                assert acc[b, :keep].tolist() == [held[b][s] for s in at_row.tolist()]
    assert evictions == 2 and dsa.dsa_get_device_status() == 0


def relative(got, want):
    return float((got.double() - want).norm() / want.norm())


@gpu
@pytest.mark.parametrize("B,T,S,n,k", [
    (8, 1, 65, 65, 0), (8, 1, 100, 100, 0), (8, 1, 190, 190, 0), (8, 1, 600, 600, 0), (8, 1, 5000, 100, 0), (2, 7, 120, 120, 0),
    (4, 1, 1024, 1024, 0), (4, 1, 1025, 1025, 0), (2, 1, 9000, 9000, 0), (8, 1, 5000, 5000, 67), (8, 1, 5000, 5000, 140),
    (2, 3, 3000, 3000, 130), (4, 1, 9000, 9000, 1024), (4, 1, 9000, 9000, 1500)])
def test_as_exact_as_fp32_products(B, T, S, n, k):
    """The weights' error in the 2-norm is that of the scores. With fp32 products and sums, each rounded to nearest, a
    score of size |z| <= 16 is off by its own last roundings (scale and difference: 2^-24 |z| each, about 5e-7 where the
    heaviest weights lie) and by the sum's; that form is computed here, and the kernel stays within half more of it, or
    within 1e-6, about 16 * 2^-24. n rows of S are visible."""
    q, kv, q_pos, kv_len = make(B, T, S, seed=S + k, lens=[n] * B)
    q_pos.fill_(n - 1)
    rows = kv[:, None, :n].expand(B, T, n, 576)
    if k:
        g = torch.Generator(device="cuda").manual_seed(k)
        idx = torch.rand((B, T, S), generator=g, device="cuda").topk(k, -1).indices.sort(-1).values.to(torch.int32).contiguous()
        rows = kv[torch.arange(B, device="cuda")[:, None, None], idx.long()]
    exact = SCALE * torch.matmul(q.double(), rows.double().transpose(-1, -2))
    lse = torch.logsumexp(exact, -1).float()
    want = torch.exp(exact - lse.double()[..., None]).sum(2)
    plain = torch.exp(SCALE * torch.matmul(q.float(), rows.float().transpose(-1, -2)) - lse[..., None]).sum(2)
    if k:
        w, _ = dsa.dsa_mla_weights_selected(q, kv, idx, lse)
    else:
        w, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    assert dsa.dsa_get_device_status() == 0
    got, base = relative(w[..., :want.shape[2]], want), relative(plain, want)
    assert got <= max(1e-6, 1.5 * base), (got, base)


@gpu
def test_queries_on_both_sides_of_the_border():
    """Queries of 1023 to 1026 visible rows in one call, then short and long ones in turn: what a query gets depends on
    its own rows alone."""
    S = 1400
    q, kv, _, kv_len = make(1, 12, S, seed=31, lens=[S])
    seen = [1023, 1024, 1025, 1026, 5, 1400, 256, 1025, 1, 1300, 1024, 1399]
    q_pos = torch.tensor([[n - 1 for n in seen]], dtype=torch.int32, device="cuda")
    rows = [[torch.arange(n, device="cuda") for n in seen]]
    lse = lse_of(q, kv, rows)
    w, _ = dsa.dsa_mla_weights(q, kv, lse, q_pos, kv_len)
    ref = reference(q, kv, lse, rows)
    for t, n in enumerate(seen):
        close(w[0, t, :n], *ref[0][t])
        assert bool((w[0, t, n:S] == 0).all())
        alone, _ = dsa.dsa_mla_weights(q[:, t:t + 1].contiguous(), kv, lse[:, t:t + 1].contiguous(),
                                       torch.tensor([[n - 1]], dtype=torch.int32, device="cuda"), kv_len)
        assert torch.equal(alone[0, 0, :S], w[0, t, :S])
    assert dsa.dsa_get_device_status() == 0
