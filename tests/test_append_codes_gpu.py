"""Which e4m3 code a rotated key is stored as.  Another than the nearest to the
64-bit quotient is one only where that lies between the two, as near to their
middle as fp32 arithmetic is off, and as rarely as that arithmetic's typical
error makes it."""
import math

import pytest
import torch

import decode_util as U

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
# Of |a| + |b| of the pair: the angle in half turns is rounded once to fp32 (2^-25, times pi), sine and cosine to one
# unit (2^-24 below 1), and two products' sum twice (2^-24 each)
TURN = 3.15 * 2.0 ** -25 + 3 * 2.0 ** -24
# The typical (root mean square) error in the same unit, the roundings being independent, in 2^-25: the angle's 0.44 pi
# on the other component (0.71 of the pair's length, which is 0.8 of |a| + |b|), 0.78; sine and cosine 1.15 on the
# length, 0.92; product, sum and quotient 0.82 on the component (0.57), three times, 0.81.  Together 1.45: 2^-24.46.
TYPICAL = 2.0 ** -24.4


@pytest.mark.parametrize("base,start,d,M", [(500000.0, 100003, 128, 16384), (10000.0, 1_000_000, 256, 8192)], ids=str)
def test_codes_of_rotated_keys(base, start, d, M):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as gg
    hkv, page = 8, 64
    g = U.gen(d)
    pages = M // page + 2
    table = torch.full((1, (start + M) // page + 1), -1, dtype=torch.int32)
    first = start // page
    table[0, first:] = torch.arange(table.shape[1] - first, dtype=torch.int32)
    pos = torch.arange(start, start + M, dtype=torch.int32)
    Z = torch.randn(M, 3 * hkv * d, generator=g).to(BF)
    kc, vc = (torch.zeros(pages, hkv, page, d, dtype=E4).cuda() for _ in range(2))
    s = torch.tensor([0.02])
    gg.coda_paged_append(Z.cuda(), pos.cuda(), table.cuda(), kc, vc, hkv, base=base, want_q=False,
                         row_seq=torch.zeros(M, dtype=torch.int32).cuda(), scale_k=s.cuda(), scale_v=s.cuda())
    assert gg.coda_get_device_status() == gg.CODA_OK
    at = table[0, (pos // page).long()].long()
    got = kc.cpu().view(torch.uint8)[at, :, (pos % page).long()].view(E4).to(U.F64)
    k = Z.view(M, 3, hkv, d)[:, 1].to(U.F64).unflatten(-1, (d // 2, 2))
    phi = pos.to(U.F64)[:, None] * torch.tensor([base ** (-2.0 * j / d) for j in range(d // 2)], dtype=U.F64)
    c, sn = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
    a, b = k[..., 0], k[..., 1]
    x = (torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2) / s.to(U.F64)).clamp(-448, 448)
    near = x.float().to(E4).to(U.F64)
    size = (a.abs() + b.abs())[..., None].expand(*a.shape, 2).flatten(-2) / s.to(U.F64)
    other = got != near
    off = size * TURN + x.abs() * 2.0 ** -23
    assert ((x - (got + near) / 2).abs() <= off)[other].all()
    assert ((got - near).abs() <= 2.0 ** -3 * near.abs().clamp(min=2.0 ** -6))[other].all()  # neighbours
    # An error e moves a value at distance t from a middle to the other code if |e| > t and its sign is the one of two:
    # half as many values change as lie within the mean |e|, which is at most the root mean square.  They are few, so
    # their number varies by its square root
    step = 2.0 ** (torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    middle = ((x / step) % 1.0 - 0.5).abs() * step
    expected = int((middle <= size * TYPICAL).sum()) / 2
    assert int(other.sum()) <= expected + 3 * math.sqrt(expected), (int(other.sum()), expected)
