"""The rotation of rows that become 8-bit codes, where the last bits of its angle show."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import serving_q8_encode_gb300 as pk
    return pk


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_angles_next_to_half_a_turn(pk, d, inter, codes):
    """(1, 0) turned by just less than half a turn: the sine is as small as what is missing, so that an error of the angle stands in it
    alone, and bf16 holds it to half a step, 2^-8 of itself. Positions are odd, so that frequencies next to half a turn stay there. Tolerance: that
    half step, a last place of the sine (2^-23) and half of one for each of two roundings beside it, and 2^-39 turns."""
    g = torch.Generator().manual_seed(d)
    gap = torch.exp2(-22 + 3 * torch.rand(d // 2, generator=g, dtype=torch.float64))      # turns
    inv = math.pi - 2 * math.pi * gap
    rope = pk.Rope(inv, interleaved=inter)
    n = 5
    q = torch.zeros(1, n, 2, d)
    (q[..., 0::2] if inter else q[..., :d // 2]).fill_(1.0)
    q = q.to(torch.bfloat16).cuda()
    k = torch.randn(1, n, 1, d, generator=g).to(torch.bfloat16).cuda()
    pos = torch.tensor([1, 3, 5, 7, 9], device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    zeros = torch.zeros(n, dtype=torch.int32, device="cuda")
    want = torch.sin(pos.double()[:, None] * 2 * math.pi * gap.cuda())[None, :, None]      # sin(odd half turn - x) = sin x
    for starts in (None, torch.arange(n + 1, dtype=torch.int32, device="cuda")):
        c = pk.PageCache.empty(1, 1, d, n, 16, "bf16", codes=codes)
        out = c.append(k, k, table, zeros, starts=starts, q=q, rope=rope, positions=pos).double()
        sin, cos = (out[..., 1::2], out[..., 0::2]) if inter else (out[..., d // 2:], out[..., :d // 2])
        assert (cos == -1).all() and c.status() == 0
        err = (sin - want).abs()
        assert (err <= want * (torch.finfo(torch.bfloat16).eps / 2 + 2.0**-22) + 2 * math.pi * 2.0**-39).all(), (err / want).max().item()
