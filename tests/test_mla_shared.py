"""dsa_mla_shared: attention over a prefix the batch shares and each sequence's own rows, against the
formula in 64 bits.

Tolerance. A score is a sum of 576 exact products accumulated in fp32: |dz| <= 576 * 2^-24 * scale *
sum |q k| =: d (the largest over the row's keys is taken), so a weight is off by a factor e^(2d); the
approximate exponential and the fp32 sums add less than 2^-18. The weights enter P V rounded to bf16
(2^-8), the output is rounded to bf16 (2^-8), pieces of a row are joined in fp32 (2^-20). Hence
|do| <= (2^-8 + 2d + 2^-16) sum p |v| + 2^-8 |o|, and |d lse| <= d + 2^-18 + 2^-22 |lse|."""
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
    #       q prefix P kv q_pos kv_len B T S scale out lse ws bytes stream
    good = [p, p, 128, p, p, p, 2, 1, 64, f(0.1), p, p, p, 1 << 30, n]

    def bad(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return dsa.lib.dsa_mla_shared(*a)

    assert bad(_6=0) == 1 and bad(_7=0) == 1 and bad(_2=-1) == 1 and bad(_8=-1) == 1
    assert bad(_2=0, _8=0) == 1                                     # no key at all
    assert bad(_2=(1 << 20) + 1) == 1 and bad(_8=(1 << 20) + 1) == 1 and bad(_6=1 << 13, _7=1 << 11) == 1
    assert bad(_9=f(0.0)) == 1 and bad(_9=f(float("nan"))) == 1
    for i in (0, 1, 3, 4, 5, 10):
        assert bad(**{f"_{i}": n}) == 1 and bad(**{f"_{i}": odd}) == 1
    assert bad(_11=odd) == 1 and bad(_12=odd) == 1
    size = dsa.dsa_mla_shared_workspace_size
    assert size(0, 1, 8, 8) == 0 and size(1, 1, 0, 0) == 0 and size(1, 1, 1, 0) > 0
    assert size(64, 1, 8192, 512) < 40 << 20                        # bounded whatever the lengths are
    assert size(4096, 128, 1 << 20, 1 << 20) == size(64, 1, 8192, 512)


def test_binding_refusals():
    q = torch.zeros(1, 1, 128, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                 # host memory
        dsa.dsa_mla_shared(q, torch.zeros(4, 576, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        dsa.dsa_mla_shared(q.float(), None)


# ------------------------------------------------------------------------------------------- GPU
def make(B, T, P, S, seed=0, lens=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    q = normal(B, T, 128, 576)
    prefix = normal(P, 576) if P else None
    if not S:
        return q, prefix, None, None, None
    kv = normal(B, S, 576)
    if lens is None:
        lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda")
    kv_len = torch.as_tensor(lens, dtype=torch.int32, device="cuda")
    q_pos = (kv_len[:, None] - T + torch.arange(T, device="cuda")).to(torch.int32)
    return q, prefix, kv, q_pos, kv_len


def check(out, lse, q, prefix, kv, q_pos, kv_len, scale=SCALE):
    B, T = q.shape[:2]
    for b in range(B):
        for t in range(T):
            keys = [prefix] if prefix is not None else []
            if kv is not None:
                seen = max(0, min(int(q_pos[b, t]) + 1, int(kv_len[b]), kv.shape[1]))
                keys.append(kv[b, :seen])
            k = torch.cat(keys).double()
            o, ls = out[b, t].double(), lse[b, t].double() if lse is not None else None
            if len(k) == 0:
                assert bool((o == 0).all()) and (ls is None or bool((ls == -torch.inf).all()))
                continue
            x = q[b, t].double()
            z = scale * x @ k.t()
            d = 576 * 2.0 ** -24 * scale * (x.abs() @ k.abs().t()).amax(-1)
            p = torch.softmax(z, -1)
            want, size = p @ k[:, :512], p @ k[:, :512].abs()
            tol = (2.0 ** -8 + 2 * d[:, None] + 2.0 ** -16) * size + 2.0 ** -8 * want.abs()
            err = (o - want).abs()
            assert bool((err <= tol).all()), (b, t, float((err - tol).max()))
            if ls is not None:
                ref = torch.logsumexp(z, -1)
                assert bool(((ls - ref).abs() <= d + 2.0 ** -18 + 2.0 ** -22 * ref.abs()).all()), (b, t)


@gpu
@pytest.mark.parametrize("B,T,P,S", [
    (1, 1, 1, 0), (2, 1, 128, 0), (1, 1, 0, 1), (2, 1, 0, 130), (3, 1, 1, 1), (2, 1, 127, 33), (5, 1, 129, 64),
    (8, 1, 1031, 256), (1, 2, 64, 96), (1, 3, 130, 200), (3, 5, 0, 161), (2, 4, 257, 31), (65, 1, 300, 40),
    (1, 1, 5000, 7), (2, 130, 70, 140), (150, 1, 140, 0)])
def test_shared(B, T, P, S):
    args = make(B, T, P, S, seed=B + T)
    out, lse = dsa.dsa_mla_shared(*args)
    assert dsa.dsa_get_device_status() == 0
    check(out, lse, *args)


@gpu
@pytest.mark.parametrize("T", [1, 2, 3])
def test_lengths_of_zero_full_and_beyond(T):
    """Sequences without an own row, with one, at tile borders, full, and lengths past the cache; with and
    without a prefix (without: rows that see nothing)."""
    lens = [0, 1, 31, 32, 33, 127, 128, 129, 255, 256, 300, 0, 0, 5]
    for P in (0, 40):
        q, prefix, kv, q_pos, kv_len = make(len(lens), T, P, 256, seed=3, lens=lens)
        q_pos[3] = -1
        q_pos[5] = 1 << 30
        q_pos[6] = -(1 << 31)
        out, lse = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
        assert dsa.dsa_get_device_status() == 0
        check(out, lse, q, prefix, kv, q_pos, kv_len)


@gpu
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("P", [0, 65])
def test_hidden_rows_may_hold_anything(T, P):
    q, prefix, kv, q_pos, kv_len = make(6, T, P, 300, seed=5, lens=[0, 7, 64, 130, 299, 300])
    clean = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
    for fill in (float("nan"), float("inf"), -3.38e38):
        dirty = kv.clone()
        for b in range(6):
            dirty[b, int(kv_len[b]):] = fill
        got = dsa.dsa_mla_shared(q, prefix, dirty, q_pos, kv_len)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # a visible NaN belongs to its own sequence
    kv[1, 3] = float("nan")
    got = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
    for b in range(6):
        if b == 1:
            assert bool(got[0][b, -1].isnan().all())
        else:
            assert torch.equal(got[0][b], clean[0][b])


@gpu
@pytest.mark.parametrize("P", [0, 200])
def test_a_row_that_only_a_later_query_sees(P):
    """A NaN or infinity there is the later query's alone, wherever in a tile the two part."""
    for n in (2, 20, 64, 65, 100, 128, 129, 200):
        q, prefix, kv, q_pos, kv_len = make(2, 2, P, 256, seed=n, lens=[n, n])
        clean = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
        for fill in (float("nan"), float("inf")):
            kv[0, n - 1, 7] = fill
            got = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
            assert torch.equal(got[0][0, 0], clean[0][0, 0]) and torch.equal(got[1][0, 0], clean[1][0, 0])
            assert torch.equal(got[0][1], clean[0][1]) and bool(got[0][0, 1].isnan().any())


@gpu
def test_queries_of_a_sequence_far_apart():
    """Positions in any order: neighbours that part in different tiles, one that sees nothing."""
    q, prefix, kv, _, kv_len = make(3, 4, 70, 400, seed=21, lens=[400, 399, 256])
    q_pos = torch.tensor([[399, 3, -1, 200], [130, 131, 64, 63], [255, 127, 128, 0]], dtype=torch.int32, device="cuda")
    for pre in (prefix, None):
        out, lse = dsa.dsa_mla_shared(q, pre, kv, q_pos, kv_len)
        check(out, lse, q, pre, kv, q_pos, kv_len)


@gpu
def test_large_scores_move_the_maximum():
    """Keys that grow along the row: the running maximum moves at every tile, by up to 2^100."""
    q, prefix, kv, q_pos, kv_len = make(3, 1, 600, 200, seed=7, lens=[200, 111, 1])
    ramp = torch.linspace(0.01, 6.0, 600, device="cuda")[:, None]
    prefix = (prefix.float() * ramp).bfloat16()
    kv = (kv.float() * 8.0).bfloat16()
    out, lse = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
    check(out, lse, q, prefix, kv, q_pos, kv_len)
    # the same keys the other way round
    out, lse = dsa.dsa_mla_shared(q, prefix.flip(0).contiguous(), kv, q_pos, kv_len)
    check(out, lse, q, prefix, kv, q_pos, kv_len)


@gpu
def test_prefix_equals_the_same_rows_kept_per_sequence():
    """The split of a context into prefix and own rows changes nothing but roundings."""
    q, prefix, kv, q_pos, kv_len = make(4, 2, 200, 100, seed=8, lens=[100, 3, 50, 77])
    out, lse = dsa.dsa_mla_shared(q, prefix, kv, q_pos, kv_len)
    whole = torch.cat([prefix.expand(4, 200, 576), kv], 1).contiguous()
    out2, lse2 = dsa.dsa_mla_shared(q, None, whole, q_pos + 200, kv_len + 200)
    check(out2, lse2, q, prefix, kv, q_pos, kv_len)
    assert bool((lse - lse2).abs().max() < 1e-4)


@gpu
def test_matches_sparse_attention_over_every_row():
    """With a short context the selection is every row: both operators compute the same attention."""
    q, _, kv, q_pos, kv_len = make(3, 1, 0, 192, seed=9, lens=[192, 100, 1])
    idx = torch.arange(192, device="cuda", dtype=torch.int32).expand(3, 1, 192)
    idx = torch.where(idx < kv_len[:, None, None], idx, -1).contiguous()
    out, lse = dsa.dsa_sparse_mla(q, kv, idx)
    check(out, lse, q, None, kv, q_pos, kv_len)
    out, lse = dsa.dsa_mla_shared(q, None, kv, q_pos, kv_len)
    check(out, lse, q, None, kv, q_pos, kv_len)


@gpu
def test_repeats_streams_graphs_workspaces():
    args = make(9, 1, 500, 90, seed=10)
    out, lse = dsa.dsa_mla_shared(*args)
    again = dsa.dsa_mla_shared(*args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])            # no order that varies
    out2, none = dsa.dsa_mla_shared(*args, want_lse=False)
    assert none is None and torch.equal(out, out2)
    ws = torch.full((dsa.dsa_mla_shared_workspace_size(9, 1, 500, 90),), 255, dtype=torch.uint8, device="cuda")
    out3, _ = dsa.dsa_mla_shared(*args, workspace=ws)                            # garbage in the scratch
    assert torch.equal(out, out3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out4, _ = dsa.dsa_mla_shared(*args, stream=side)
    out5, _ = dsa.dsa_mla_shared(*args)                                          # two calls at once
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, out4) and torch.equal(out, out5)
    # captured: lengths are read at replay, so a grown cache needs no new capture
    q, prefix, kv, q_pos, kv_len = args
    res, rl = torch.empty_like(out), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_mla_shared(*args, out=res, lse=rl, workspace=ws)
    for n in (0, 17, 90):
        kv_len.fill_(n)
        q_pos.fill_(n - 1)
        g.replay()
        check(res, rl, q, prefix, kv, q_pos, kv_len)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_mla_shared(*args, workspace=ws[:1024])
    assert e.value.code == 6
    for bad in (dict(q=q[..., :575].contiguous()), dict(prefix=prefix[:, :512].contiguous()), dict(kv=kv[:8].contiguous()),
                dict(q_pos=q_pos[:8].contiguous()), dict(kv_len=kv_len.long()), dict(kv=None), dict(out=out[:8]),
                dict(lse=lse.half()), dict(prefix=prefix.cpu()), dict(q=q.transpose(0, 1))):
        with pytest.raises((ValueError, TypeError)):
            dsa.dsa_mla_shared(**{**dict(q=q, prefix=prefix, kv=kv, q_pos=q_pos, kv_len=kv_len), **bad})


@gpu
def test_own_rows_past_32_bit_offsets():
    """A cache of more than 2^31 elements; the last sequence's rows lie beyond."""
    B, S = 4, 940000
    kv = torch.zeros((B, S, 576), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() > 1 << 31
    q, prefix, _, _, _ = make(B, 1, 50, 0, seed=12)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = torch.tensor([3, 150, 0, 201], dtype=torch.int32, device="cuda")
    kv[:, :201] = torch.randn((B, 201, 576), generator=g, device="cuda").bfloat16()
    kv[:, 201:205] = float("nan")
    out, lse = dsa.dsa_mla_shared(q, prefix, kv, lens[:, None] - 1, lens)
    check(out, lse, q, prefix, kv, lens[:, None] - 1, lens)


@gpu
@pytest.mark.parametrize("B,T,P,S", [(1000, 1, 70, 64), (3, 301, 70, 150), (901, 1, 0, 140), (1, 1601, 130, 20)])
def test_more_units_than_threads_plan_at_once(B, T, P, S):
    """Over 768 tokens a thread plans several units, and cuts fall between and inside them; sequences without a row
    among them, and (without a prefix) whole units that see nothing."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, S + 1, (B,), generator=g)
    lens[::3] = 0
    lens[40:60] = 0
    lens[-1] = S
    args = make(B, T, P, S, seed=13, lens=lens.cuda())
    out, lse = dsa.dsa_mla_shared(*args)
    assert dsa.dsa_get_device_status() == 0
    check(out, lse, *args)
    again = dsa.dsa_mla_shared(*args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
