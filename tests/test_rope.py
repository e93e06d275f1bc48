"""dsa_rope and dsa_rope_freqs: rotary positions on part of a head, against the rotation in 64 bits.

Tolerance of y = u cos - v sin: the angle is rounded once to fp32 (at most half a turn, pi 2^-25) and
sincospi is good to two steps of 2^-24, together under 2^-22; the scale, the product and the sum add
three roundings of 2^-24. So |dy| <= 2^-21 |scale| (|u| + |v|), plus half a step of the output type."""
import ctypes
import math

import pytest
import torch

import __graft_entry__

__graft_entry__._build_module().build()
import sparse_attention_keys_b200 as dsa  # noqa: E402

gpu = pytest.mark.gpu


def radians(freqs):
    """The 2^-64 turns of dsa_rope_freqs as float64 radians per position."""
    return torch.tensor([(int(f) & (2 ** 64 - 1)) / 2 ** 64 * 2 * math.pi for f in freqs], dtype=torch.float64)


def rotated(x, pos, freqs, offset, interleaved, inverse=False, scale=1.0):
    """x [rows, heads, dim] float64 -> (rotated, |u| + |v| of each element's pair)."""
    n = len(freqs)
    # the angle modulo a turn in whole numbers: exact at any position
    turns = [[(int(p) * (int(f) & (2 ** 64 - 1))) % 2 ** 64 / 2 ** 64 for f in freqs] for p in pos]
    a = 2 * math.pi * torch.tensor(turns, dtype=torch.float64, device=x.device)[:, None] * (-1 if inverse else 1)
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    first = slice(offset, offset + 2 * n, 2) if interleaved else slice(offset, offset + n)
    second = slice(offset + 1, offset + 2 * n, 2) if interleaved else slice(offset + n, offset + 2 * n)
    u, v = x[..., first], x[..., second]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = u * c - v * s, u * s + v * c
    size[..., first] = size[..., second] = (u.abs() + v.abs()) * abs(scale)
    return y, size


def check(got, x, pos, freqs, offset, interleaved, inverse=False, scale=1.0):
    y, size = rotated(x.double(), pos, freqs, offset, interleaved, inverse, scale)
    half_step = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half_step * 2     # half a step below the normal range
    # features outside the rotary part are copied, bit for bit
    n = 2 * len(freqs)
    assert torch.equal(got[..., :offset], x[..., :offset]) and torch.equal(got[..., offset + n:], x[..., offset + n:])
    err = (got.double() - y).abs()
    tol = half_step * y.abs() + (1 + half_step) * 2.0 ** -21 * size + tiny
    tol[size == 0] = 0
    assert bool((err <= tol).all()), f"worst {(err - tol).max():.3g}"


# ------------------------------------------------------------------------------------------- CPU
@pytest.mark.parametrize("pairs,theta,factor,original", [(32, 1e4, 40.0, 4096), (64, 5e5, 1.0, 0), (16, 1e4, 8.0, 0),
                                                         (1, 2.0, 1.0, 0), (128, 1e6, 4.0, 32768), (7, 10.0, 3.0, 100000)])
def test_freqs_follow_the_formula(pairs, theta, factor, original):
    got = radians(dsa.dsa_rope_freqs(pairs, theta=theta, factor=factor, original_len=original))
    dim = 2 * pairs
    for i in range(pairs):
        f = theta ** (-2.0 * i / dim)
        slowed = 1.0
        if original:
            def corr(n):
                return dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(theta))
            low, high = max(math.floor(corr(32.0)), 0), min(math.ceil(corr(1.0)), dim - 1)
            if high <= low:
                high = low + 0.001
            slowed = min(max((i - low) / (high - low), 0.0), 1.0)
        want = f if factor == 1.0 else f * (1 - slowed) + f / factor * slowed
        # half a unit of 2^-64 turns, and float64's own error
        assert abs(float(got[i]) - want) <= 2 * math.pi * 2.0 ** -65 + 1e-14 * want, i


def test_freqs_match_the_model_table():
    """theta 1e4, factor 40, 4096 positions: the frequencies behind dsa_rope_table (which rounds the
    angle to fp32: 2^-24 of it)."""
    table = dsa.dsa_rope_table(600).double()
    a = torch.arange(600)[:, None] * radians(dsa.dsa_rope_freqs(32, factor=40.0, original_len=4096))
    tol = 2.0 ** -23 * a + 2.0 ** -23
    assert bool(((table[..., 0] - torch.cos(a)).abs() <= tol).all())
    assert bool(((table[..., 1] - torch.sin(a)).abs() <= tol).all())


def test_freqs_refusals():
    for bad in ({"theta": 1.0}, {"theta": math.inf}, {"factor": 0.5}, {"factor": math.nan}, {"original_len": -1},
                {"beta_slow": 0.0}, {"beta_fast": 1.0}):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_rope_freqs(8, **bad)
    for pairs in (0, -3):
        with pytest.raises(ValueError):
            dsa.dsa_rope_freqs(pairs)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope_freqs(2049)


def test_abi_refusals():
    """Rejected on the host before any launch (no device here)."""
    p, odd, n = ctypes.c_void_p(64), ctypes.c_void_p(65), None
    f = ctypes.c_float
    #       x dtype rows heads xr xh dim off pairs pos freqs scale flags out or oh stream
    good = [p, 1, 4, 2, 256, 128, 128, 0, 32, p, p, f(1.0), 0, ctypes.c_void_p(4096), 256, 128, n]
    call = dsa.lib.dsa_rope

    def bad(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return call(*a)

    assert bad(_2=0) == 0                                          # no rows: nothing to do
    assert bad(_1=3) == 1 and bad(_2=-1) == 1 and bad(_3=0) == 1 and bad(_3=4097) == 1
    assert bad(_6=0) == 1 and bad(_6=4097) == 1
    assert bad(_7=-1) == 1 and bad(_7=65) == 1 and bad(_8=0) == 1 and bad(_8=65) == 1
    assert bad(_8=0x7fffffff) == 1                                 # 2 * pairs past int32
    assert bad(_11=f(math.inf)) == 1 and bad(_12=0x40) == 1
    assert bad(_0=n) == 1 and bad(_9=n) == 1 and bad(_10=n) == 1 and bad(_13=n) == 1
    assert bad(_0=odd) == 1 and bad(_13=odd) == 1 and bad(_9=ctypes.c_void_p(66)) == 1 and bad(_10=ctypes.c_void_p(68)) == 1
    assert bad(_4=-1) == 1 and bad(_14=-1) == 1
    assert bad(_14=0) == 1 and bad(_15=64) == 1 and bad(_14=255) == 1   # outputs that would coincide
    assert bad(_13=p, _14=512) == 1                                # in place with other strides


def test_binding_refusals():
    freqs = dsa.dsa_rope_freqs(2)
    with pytest.raises(TypeError):
        dsa.dsa_rope(torch.zeros(1, 4, dtype=torch.float64), torch.zeros(1, dtype=torch.int32), freqs)
    with pytest.raises(ValueError):                                # host tensors
        dsa.dsa_rope(torch.zeros(1, 4), torch.zeros(1, dtype=torch.int32), freqs)


# ------------------------------------------------------------------------------------------- GPU
def make(rows, heads, dim, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, heads, dim), generator=g, device="cuda").to(dtype)


def positions(rows, seed=1):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-(1 << 20), 1 << 20, (rows,), generator=g, dtype=torch.int32)
    pos[:3] = torch.tensor([0, 2 ** 31 - 1, -2 ** 31])[:min(rows, 3)]
    return pos


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,offset,pairs", [
    (1, 1, 2, 0, 1), (3, 1, 64, 0, 32), (5, 128, 192, 128, 32), (1, 4096, 8, 0, 4), (67, 3, 33, 5, 9),
    (2, 7, 4096, 0, 2048), (130, 2, 128, 0, 32), (9, 1, 576, 512, 32), (33, 5, 24, 8, 8), (700, 1, 16, 8, 4)])
def test_rope(dtype, interleaved, rows, heads, dim, offset, pairs):
    x, pos, freqs = make(rows, heads, dim, dtype), positions(rows), dsa.dsa_rope_freqs(pairs, factor=4.0, original_len=512)
    got = dsa.dsa_rope(x, pos.cuda(), freqs.cuda(), offset=offset, interleaved=interleaved)
    check(got, x, pos, freqs, offset, interleaved)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_strides_and_places(interleaved):
    """A slice of wider rows, heads outermost, an odd column, in place, and a broadcast input."""
    freqs = dsa.dsa_rope_freqs(32)
    f = freqs.cuda()
    pos = positions(11)
    p = pos.cuda()
    wide = make(11, 1, 640, torch.bfloat16).squeeze(1)
    for col in (512, 513):                                          # 16-byte aligned, and not
        x = wide[:, col:col + 64]
        check(dsa.dsa_rope(x, p, f, interleaved=interleaved)[:, None], x[:, None], pos, freqs, 0, interleaved)
        # in place: the rest of the rows stays
        here = wide.clone()
        dsa.dsa_rope(here[:, col:col + 64], p, f, interleaved=interleaved, out=here[:, col:col + 64])
        check(here[:, None, col:col + 64], x[:, None], pos, freqs, 0, interleaved)
        here[:, col:col + 64] = x
        assert torch.equal(here, wide)
        # into the neighbouring columns of the same rows
        dsa.dsa_rope(here[:, col:col + 64], p, f, interleaved=interleaved, out=here[:, 100:164])
        check(here[:, None, 100:164], x[:, None], pos, freqs, 0, interleaved)
    x = make(6, 11, 64, torch.float32).transpose(0, 1)              # heads outermost
    out = torch.full((6, 11, 72), 7.0, device="cuda")
    dsa.dsa_rope(x, p, f, interleaved=interleaved, out=out.transpose(0, 1)[..., 8:])
    check(out.transpose(0, 1)[..., 8:], x, pos, freqs, 0, interleaved)
    assert bool((out[..., :8] == 7.0).all())
    x = make(1, 3, 64, torch.float16).expand(11, 3, 64)             # one row at eleven positions
    check(dsa.dsa_rope(x, p, f, interleaved=interleaved), x, pos, freqs, 0, interleaved)
    assert dsa.dsa_rope(make(0, 3, 64, torch.float32), p[:0], f).shape == (0, 3, 64)


@gpu
def test_rope_offsets_past_32_bits():
    """Rows whose elements lie more than 2^31 apart."""
    buf = torch.empty((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, 2, 64), ((1 << 31) + 128, 64, 1))
    x.copy_(make(2, 2, 64, torch.bfloat16))
    freqs, pos = dsa.dsa_rope_freqs(32), positions(2)
    want = x.clone()
    dsa.dsa_rope(x, pos.cuda(), freqs.cuda(), out=x)
    check(x, want, pos, freqs, 0, False)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """inverse=True is the gradient: the formula's (64 bits), and central differences of the rotation."""
    freqs, pos, scale = dsa.dsa_rope_freqs(8), positions(5), 1.25
    x, g = make(5, 3, 24, torch.float32), make(5, 3, 24, torch.float32, seed=9)
    kw = dict(offset=4, interleaved=interleaved, scale=scale)
    gx = dsa.dsa_rope(g, pos.cuda(), freqs.cuda(), inverse=True, **kw)
    xd = x.double().requires_grad_()
    y, _ = rotated(xd, pos, freqs, 4, interleaved, scale=scale)
    want, = torch.autograd.grad((y * g.double()).sum(), xd)
    size = rotated(g.double().abs(), pos, freqs, 4, interleaved, scale=scale)[1]
    assert bool(((gx.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -21 * size + 1e-30).all())
    # the rotation is linear: differences of the kernel itself, over a step of 1 (no truncation error)
    d = make(5, 3, 24, torch.float32, seed=11)
    y0, y1 = (dsa.dsa_rope(x + s * d, pos.cuda(), freqs.cuda(), **kw).double() for s in (-1.0, 1.0))
    directional = ((y1 - y0) / 2 * g.double()).sum()
    # each output is off by 2^-21 (|u| + |v|) scale and a rounding, each input sum by a rounding
    bound = ((x.abs() + d.abs()).sum(-1, keepdim=True) * scale * 2.0 ** -20 * g.abs()).double().sum()
    assert abs(float(directional - (gx.double() * d.double()).sum())) <= float(bound)


@gpu
def test_rope_moves_a_key_by_the_difference():
    """Keys rotated at p, then by q - p, are keys rotated at q: how cached rows change position."""
    freqs = dsa.dsa_rope_freqs(32, factor=40.0, original_len=4096)
    f = freqs.cuda()
    cache = make(1, 50, 576, torch.float32).squeeze(0)
    p, q = positions(50, 3) >> 12, positions(50, 4) >> 12
    here = cache.clone()
    for step in (p, q - p):
        dsa.dsa_rope(here, step.cuda(), f, offset=512, interleaved=True, out=here)
    y, size = rotated(cache[:, None].double(), q, freqs, 512, True)
    # two rotations in fp32, each within 2^-21 (|u| + |v|); the first's sum is at most sqrt 2 of it
    assert bool(((here[:, None].double() - y).abs() <= 3 * 2.0 ** -21 * size + 2.0 ** -23 * y.abs()).all())
    assert torch.equal(here[:, :512], cache[:, :512])


@gpu
def test_rope_streams_graphs_and_refusals():
    freqs, pos = dsa.dsa_rope_freqs(32).cuda(), positions(40)
    x = make(40, 2, 64, torch.bfloat16)
    want = dsa.dsa_rope(x, pos.cuda(), freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_rope(x, pos.cuda(), freqs, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    p, out = pos.cuda(), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_rope(x, p, freqs, out=out)
    x.mul_(2.0)                                                     # exact in bf16
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2.0 * want)
    for bad in (dict(x=x[..., ::2]), dict(pos=p[:39]), dict(pos=p.long()), dict(freqs=freqs.cpu()), dict(offset=1),
                dict(offset=-2), dict(out=out[:39]), dict(out=out.float()), dict(out=x[:, :1].expand(40, 2, 64))):
        with pytest.raises((ValueError, TypeError)):
            dsa.dsa_rope(**{**dict(x=x, pos=p, freqs=freqs), **bad})
    buf = make(41, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError):                                 # one row further: overlaps its input
        dsa.dsa_rope(buf[:40], p, freqs, out=buf[1:])
    assert dsa.dsa_get_device_status() == 0
