"""dsa_cache_evict: which rows stay, and where each ends up, exactly as defined."""
import ctypes
import math

import pytest
import torch

import __graft_entry__

__graft_entry__._build_module().build()
import sparse_attention_keys_b200 as dsa  # noqa: E402

gpu = pytest.mark.gpu


def plan(acc, pos, n, keep, recent, sinks):
    """src of one sequence: acc, pos as lists."""
    n = max(0, min(n, len(acc)))
    if n <= keep:
        return list(range(n)) + [-1] * (keep - n)
    newest = max(pos[:n])
    safe = [pos[r] > newest - recent or pos[r] < sinks for r in range(n)]
    # NaN below every weight
    ranked = sorted(range(n), key=lambda r: (not safe[r], math.isnan(acc[r]), -acc[r] if acc[r] == acc[r] else 0.0, r))
    kept = sorted(ranked[:keep])
    movers = iter([r for r in kept if r >= keep])
    there = set(kept)
    return [i if i in there else next(movers) for i in range(keep)]


def test_abi_refusals():
    p, odd, n = ctypes.c_void_p(64), ctypes.c_void_p(65), None
    #       acc pos len B S keep recent sinks kv k8 ks acc_out pos_out len_out src ws bytes stream
    good = [p, p, p, 2, 64, 32, 4, 1, p, p, p, p, p, p, p, p, 1 << 30, n]

    def bad(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return dsa.lib.dsa_cache_evict(*a)

    assert bad(_3=0) == 1 and bad(_3=65536) == 1 and bad(_4=0) == 1 and bad(_4=(1 << 20) + 1) == 1
    assert bad(_5=0) == 1 and bad(_6=-1) == 1 and bad(_7=-1) == 1
    assert bad(_9=n) == 1 and bad(_10=n) == 1                       # codes without scales, scales without codes
    for i in (0, 1, 2, 11, 12, 13):
        assert bad(**{f"_{i}": n}) == 1 and bad(**{f"_{i}": odd}) == 1
    for i in (8, 9, 10, 14, 15):
        assert bad(**{f"_{i}": odd}) == 1
    size = dsa.dsa_cache_evict_workspace_size
    assert size(0, 8, 4) == 0 and size(1, 8, 0) == 0
    assert size(2, 64, 32) == 2 * (1 + 2 * 32) * 4 + 8 and size(1, 64, 100) == 16


def test_binding_refusals():
    acc = torch.zeros(1, 8)
    with pytest.raises(ValueError):
        dsa.dsa_cache_evict(acc, acc.int(), torch.zeros(1, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        dsa.dsa_cache_evict(acc.double(), acc.int(), torch.zeros(1, dtype=torch.int32), 4)


# ------------------------------------------------------------------------------------------- GPU
def state(B, S, seed=0, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    acc = torch.rand((B, S), generator=g, device="cuda")
    if ties:
        acc = (acc * 4).floor() / 4
    pos = torch.rand((B, S), generator=g, device="cuda").argsort(1).to(torch.int32)
    kv = torch.randint(-32768, 32767, (B, S, 576), generator=g, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    k8 = torch.randint(0, 256, (B, S, 128), generator=g, device="cuda", dtype=torch.uint8)
    ks = torch.rand((B, S), generator=g, device="cuda")
    return acc, pos, kv, k8, ks


def check(acc, pos, lens, keep, recent=0, sinks=0, caches=True, seed=0):
    """Out of place for the state, in place for the caches, then in place for all."""
    B, S = acc.shape
    _, _, kv, k8, ks = state(B, S, seed=seed + 100)
    if not caches:
        kv = k8 = ks = None
    kv_len = torch.as_tensor(lens, dtype=torch.int32, device="cuda")
    want = torch.tensor([plan(a, p, int(n), keep, recent, sinks)
                         for a, p, n in zip(acc.tolist(), pos.tolist(), lens)], device="cuda")
    live = want >= 0
    bi = torch.arange(B, device="cuda")[:, None].expand_as(want)

    def expect(t):                                     # rows behind the new length stay as they were
        e = t.clone()
        rows = torch.arange(want.shape[1], device="cuda").expand_as(want)
        e[bi[live], rows[live]] = t[bi[live], want[live]]
        return e

    old = [None if t is None else t.clone() for t in (kv, k8, ks)]
    acc_out, pos_out = torch.full_like(acc, -7.0), torch.full_like(pos, -7)
    len_out = torch.empty_like(kv_len)
    r = dsa.dsa_cache_evict(acc, pos, kv_len, keep, recent=recent, sinks=sinks, kv=kv, k8=k8, k_scale=ks,
                            acc_out=acc_out, pos_out=pos_out, kv_len_out=len_out)
    assert torch.equal(r[3].long(), want)
    assert len_out.tolist() == [min(max(0, min(n, S)), keep) for n in lens]
    for new, before in zip((kv, k8, ks), old):
        if new is not None:
            same = new.view(torch.int16) if new.dtype == torch.bfloat16 else new
            ref = expect(before)
            assert torch.equal(same, ref.view(torch.int16) if new.dtype == torch.bfloat16 else ref)
    ref_acc, ref_pos = torch.full_like(acc, -7.0), torch.full_like(pos, -7)
    rows = torch.arange(want.shape[1], device="cuda").expand_as(want)
    ref_acc[bi[live], rows[live]] = acc[bi[live], want[live]]
    ref_pos[bi[live], rows[live]] = pos[bi[live], want[live]]
    assert torch.equal(acc_out.view(torch.int32), ref_acc.view(torch.int32)) and torch.equal(pos_out, ref_pos)
    ea, ep = expect(acc), expect(pos)
    acc, pos = acc.clone(), pos.clone()
    dsa.dsa_cache_evict(acc, pos, kv_len, keep, recent=recent, sinks=sinks)
    assert torch.equal(acc.view(torch.int32), ea.view(torch.int32)) and torch.equal(pos, ep)
    assert torch.equal(kv_len, len_out)
    assert dsa.dsa_get_device_status() == 0


@gpu
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("B,S,keep,recent,sinks", [
    (1, 1, 1, 0, 0), (1, 2, 1, 0, 0), (2, 33, 32, 3, 1), (3, 100, 7, 0, 0), (5, 1000, 999, 100, 4), (2, 2304, 2048, 128, 4),
    (9, 2049, 64, 64, 0), (1, 16385, 5000, 700, 16), (3, 700, 350, 0, 350)])
def test_evict(B, S, keep, recent, sinks, ties):
    acc, pos, _, _, _ = state(B, S, seed=S, ties=ties)
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, S + 1, (B,), generator=g).tolist()
    lens[0] = S
    check(acc, pos, lens, keep, recent, sinks, caches=B * S < 20000, seed=S)


@gpu
@pytest.mark.parametrize("lens", [[0, 1, 4, 5], [8, 9, 100, -3], [7, 6, 1 << 30, 2]])
def test_lengths(lens):
    """Nothing to give up, one row over, empty, and lengths outside the cache."""
    acc, pos, _, _, _ = state(4, 8, seed=1)
    check(acc, pos, lens, 5, 2, 1)
    check(acc, pos, lens, 8)
    check(acc, pos, lens, 20, 3, 0)                    # a budget larger than the cache


@gpu
def test_special_weights():
    """Infinities, NaN, both zeros and denormals; every row equal; every row protected."""
    vals = [float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-40, -1e-40, 3.4e38, -3.4e38, 1.0, -1.0]
    acc = torch.tensor([vals * 6], device="cuda")
    pos = torch.arange(66, device="cuda", dtype=torch.int32).flip(0)[None].contiguous()
    for keep in (1, 5, 7, 20, 40, 55, 60, 65):
        check(acc, pos, [66], keep)
        check(acc, pos, [61], keep, 5, 2)
    check(torch.ones_like(acc), pos, [66], 30)
    check(acc, pos, [66], 30, 66, 0)                   # all protected: the heaviest of them
    check(acc, pos, [66], 30, 1 << 30, 1 << 30)
    check(acc, pos - (1 << 31), [66], 30, 4, 0)        # positions at the bottom of the range


@gpu
@pytest.mark.parametrize("B,S", [(1, 131072), (2, 140000), (1, 300001)])
def test_long_sequences(B, S):
    """Rows over a whole cluster; the last sizes do not fit its shared memory."""
    acc, pos, _, _, _ = state(1, 8, seed=S)
    g = torch.Generator(device="cuda").manual_seed(S)
    acc = (torch.rand((B, S), generator=g, device="cuda") * 50000).floor()
    pos = torch.arange(S, device="cuda", dtype=torch.int32).expand(B, S).contiguous()
    check(acc, pos, [S - 1] * B, 50001, 1000, 4, caches=False)


@gpu
def test_again_and_again_with_graph_and_streams():
    """Append, evict, append: one captured call; and two calls at once on two streams."""
    B, S, keep, recent = 3, 96, 64, 8
    acc, pos, kv, k8, ks = state(B, S, seed=4)
    pos = torch.arange(S, device="cuda", dtype=torch.int32).expand(B, S).contiguous()
    kv_len = torch.full((B,), S, dtype=torch.int32, device="cuda")
    src = torch.empty((B, keep), dtype=torch.int32, device="cuda")
    ws = torch.empty(dsa.dsa_cache_evict_workspace_size(B, S, keep), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_cache_evict(acc, pos, kv_len, keep, recent=recent, kv=kv, k8=k8, k_scale=ks, src=src, workspace=ws)
    assert bool((kv_len == S).all())
    for step in range(3):
        want = [plan(a, p, S, keep, recent, 0) for a, p in zip(acc.tolist(), pos.tolist())]
        rows = [torch.stack([t[b][w] for b, w in enumerate(want)]) for t in (kv.view(torch.int16), k8, ks, acc, pos)]
        g.replay()
        assert src.tolist() == want and kv_len.tolist() == [keep] * B
        for t, r in zip((kv.view(torch.int16), k8, ks, acc, pos), rows):
            assert torch.equal(t[:, :keep], r)
        acc[:, keep:] = torch.rand((B, S - keep), device="cuda")
        pos[:, keep:] = pos.max() + 1 + torch.arange(S - keep, device="cuda", dtype=torch.int32)
        kv_len.fill_(S)
    side = torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for s in (None, side):
        outs.append(dsa.dsa_cache_evict(acc, pos, kv_len, keep, acc_out=torch.empty_like(acc),
                                        pos_out=torch.empty_like(pos), kv_len_out=torch.empty_like(kv_len), stream=s))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][3], outs[1][3]) and torch.equal(outs[0][0][:, :keep], outs[1][0][:, :keep])


@gpu
def test_refusals_on_the_device():
    acc, pos, kv, k8, ks = state(2, 16)
    n = torch.full((2,), 16, dtype=torch.int32, device="cuda")
    good = dict(acc=acc, pos=pos, kv_len=n, keep=8)
    for bad in (dict(keep=0), dict(pos=pos[:1]), dict(kv_len=n.long()), dict(kv=kv[:, :15].contiguous()), dict(k8=k8),
                dict(k_scale=ks), dict(acc_out=acc[:1]), dict(src=torch.empty((2, 9), dtype=torch.int32, device="cuda")),
                dict(pos=pos.cpu()), dict(acc=acc.t())):
        with pytest.raises((ValueError, TypeError)):
            dsa.dsa_cache_evict(**{**good, **bad})
    for bad in (dict(recent=-1), dict(sinks=-1), dict(workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_cache_evict(**{**good, **bad})


@gpu
@pytest.mark.parametrize("B,S,keep", [(2, 5000, 1800), (1, 140000, 70001), (1, 140000, 9)])
def test_ties_across_every_warp_and_part_of_the_state_in_place(B, S, keep):
    """Equal weights everywhere, so that the lowest rows stay; and positions alone written elsewhere."""
    acc = torch.full((B, S), 0.5, device="cuda")
    acc[:, ::7] = 0.25
    pos = torch.arange(S, device="cuda", dtype=torch.int32).flip(0).expand(B, S).contiguous()
    kv_len = torch.full((B,), S, dtype=torch.int32, device="cuda")
    want = [plan(a, p, S, keep, 3, 0) for a, p in zip(acc.tolist(), pos.tolist())]
    rows = [torch.stack([t[b][w] for b, w in enumerate(want)]) for t in (acc, pos)]
    before, pos_out = pos.clone(), torch.full_like(pos, -7)
    _, _, n, src = dsa.dsa_cache_evict(acc, pos, kv_len, keep, recent=3, pos_out=pos_out)
    assert src.tolist() == want and n.tolist() == [keep] * B
    assert torch.equal(acc[:, :keep], rows[0]) and torch.equal(pos_out[:, :keep], rows[1])
    assert torch.equal(pos, before) and bool((pos_out[:, keep:] == -7).all())
    assert dsa.dsa_get_device_status() == 0


@gpu
def test_a_budget_of_every_int():
    """The largest budget there is: nothing to give up, and all of src behind the rows is -1."""
    keep = (1 << 31) - 1
    acc, pos, _, _, _ = state(1, 8, seed=2)
    n = torch.tensor([6], dtype=torch.int32, device="cuda")
    src = torch.zeros((1, keep), dtype=torch.int32, device="cuda")
    assert dsa.dsa_cache_evict_workspace_size(1, 8, keep) == 16
    out = [torch.full_like(acc, -7.0), torch.full_like(pos, -7), torch.empty_like(n)]
    dsa.dsa_cache_evict(acc, pos, n, keep, acc_out=out[0], pos_out=out[1], kv_len_out=out[2], src=src)
    assert dsa.dsa_get_device_status() == 0
    assert out[2].tolist() == [6] and src[0, :6].tolist() == list(range(6))
    assert torch.equal(out[0][0, :6], acc[0, :6]) and torch.equal(out[1][0, :6], pos[0, :6])
    assert bool((out[0][0, 6:] == -7.0).all()) and bool((out[1][0, 6:] == -7).all())
    assert all(bool((c == -1).all()) for c in src[0, 6:].split(1 << 28))


@gpu
@pytest.mark.parametrize("S", [131071, 131073])
def test_at_the_register_capacity(S):
    """Eight CTAs hold 131072 rows in registers; from one more on every pass reads them again."""
    acc = torch.rand((1, S), generator=torch.Generator(device="cuda").manual_seed(S), device="cuda")
    acc = (acc * 1000).floor()
    pos = torch.arange(S, device="cuda", dtype=torch.int32)[None].contiguous()
    for n in (S, S - 1):
        check(acc, pos, [n], 60001, 500, 4, caches=False)
