"""Where dsa_rope may write when x and out share memory: told from the strides, against the elements themselves."""
import random

import pytest
import torch

import __graft_entry__

__graft_entry__._build_module().build()
import sparse_attention_keys_b200 as dsa  # noqa: E402


def elements(at, rows, heads, dim, row, head):
    return {at + r * row + h * head + i for r in range(rows) for h in range(heads) for i in range(dim)}


def test_whatever_counts_as_apart_is():
    rng = random.Random(5)
    apart = 0
    for _ in range(6000):
        rows, heads, dim = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 4)
        xr, xh = rng.randint(0, 24), rng.randint(0, 24)
        yr, yh = (xr, xh) if rng.random() < 0.7 else (rng.randint(0, 24), rng.randint(0, 24))
        d = rng.randint(-40, 40)
        if dsa._rope_apart(d, rows, heads, dim, xr, xh, yr, yh):
            apart += 1
            assert not elements(0, rows, heads, dim, xr, xh) & elements(d, rows, heads, dim, yr, yh)
    assert apart > 1000


@pytest.mark.parametrize("name,d,rows,heads,dim,strides", [
    ("other columns of the same rows", 100, 40, 1, 64, (640, 64, 640, 64)),
    ("columns before them", -100, 40, 1, 64, (640, 64, 640, 64)),
    ("the other half of each row's heads", 8 * 64, 40, 8, 64, (16 * 64, 64, 16 * 64, 64)),
    ("heads outermost, other columns", 64, 40, 6, 64, (192, 40 * 192, 192, 40 * 192)),
    ("every other head", 64, 40, 8, 64, (16 * 64, 128, 16 * 64, 128)),
    ("heads outermost, the rows behind", 40 * 64, 40, 6, 64, (64, 80 * 64, 64, 80 * 64)),
    ("every other row", 64, 40, 1, 64, (128, 64, 128, 64)),
    ("behind it", 40 * 64, 40, 1, 64, (64, 64, 64, 64)),
])
def test_places_that_do_not_meet(name, d, rows, heads, dim, strides):
    xr, xh, yr, yh = strides
    assert not elements(0, rows, heads, dim, xr, xh) & elements(d, rows, heads, dim, yr, yh)
    assert dsa._rope_apart(d, rows, heads, dim, xr, xh, yr, yh)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_into_the_same_buffer(interleaved):
    """Heads outermost into other columns, and every other head into its neighbour: the same bits as into a new tensor."""
    freqs = dsa.dsa_rope_freqs(16).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    buf = torch.randn((4, 9, 96), generator=g, device="cuda").bfloat16()
    x, out = buf.transpose(0, 1)[..., :32], buf.transpose(0, 1)[..., 48:80]
    want, rest = dsa.dsa_rope(x, pos, freqs, interleaved=interleaved), buf.clone()
    dsa.dsa_rope(x, pos, freqs, interleaved=interleaved, out=out)
    assert torch.equal(out, want)
    rest[..., 48:80] = want.transpose(0, 1)
    assert torch.equal(buf, rest)
    buf = torch.randn((9, 8, 32), generator=g, device="cuda")
    want, rest = dsa.dsa_rope(buf[:, ::2], pos, freqs, interleaved=interleaved), buf.clone()
    dsa.dsa_rope(buf[:, ::2], pos, freqs, interleaved=interleaved, out=buf[:, 1::2])
    rest[:, 1::2] = want
    assert torch.equal(buf, rest)
    for bad in (buf[:, 1:5], buf[:, 2:6]):                          # heads that are still to be read
        with pytest.raises(ValueError, match="overlap"):
            dsa.dsa_rope(buf[:, :4], pos, freqs, out=bad)
    assert dsa.dsa_get_device_status() == 0
