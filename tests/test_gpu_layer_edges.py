"""Edges of the layer operators on the GPU: 8-bit values that lie on a tie, gates that grow, packed batches with rows
of no sequence, and the shapes and chains behind them, against the plain 64-bit forms."""
import pytest
import torch

import gated_deltanet_chunked_04_amd as gdn
from oracle import layer as ref
from test_gpu_layer import close, cu_dev, cuda, owned, packed, rnd, scan_inputs

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ---- RMS norm -----------------------------------------------------------------------------------


@pytest.mark.parametrize("rows,D", [(40, 5), (200, 64), (200, 300), (200, 512), (60, 2047), (30, 9000), (10, 20000), (6, 33001)])
def test_8_bit_values_are_the_nearest_quotients(rows, D, gpu_lib):
    """y / scale to nearest even, formed from the fp32 y: a call in the input's type gives that y, and the quotients of
    small whole numbers lie on 8-bit ties often."""
    gen = torch.Generator().manual_seed(D)
    x = torch.randint(-120, 121, (rows, D), generator=gen).float()
    x[::2] = torch.randn(len(x[::2]), D, generator=gen)
    w = torch.randint(1, 9, (D,), generator=gen).float() / 8
    y = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda())[0].cpu()
    for quant, G in (("row", D), ("group", 128)):
        q, _, scale = gdn.gdn_rmsnorm_fwd(x.cuda(), w.cuda(), quant=quant)
        want = (y / scale.cpu().repeat_interleave(G, 1)[:, :D]).clamp(-448, 448).to(torch.float8_e4m3fn)
        bad = q.cpu().view(torch.uint8) != want.view(torch.uint8)
        # (a zero may carry either sign)
        bad &= (q.cpu().float() != 0) | (want.float() != 0)
        assert not bad.any(), (quant, int(bad.sum()), bad.numel())


def test_8_bit_values_beside_an_infinity(gpu_lib):
    """Where y overflows to infinity its scale is infinite, the values beside it 0 / inf = 0, itself NaN."""
    for D in (5, 64, 300, 40000):
        x, w = torch.ones(2, D).cuda(), torch.ones(D).cuda()
        w[3] = float("inf")
        for quant in ("row", "group"):
            q, _, scale = gdn.gdn_rmsnorm_fwd(x, w, quant=quant)
            q = q.float().cpu()
            assert torch.isinf(scale[:, 0]).all() and torch.isnan(q[:, 3]).all()
            assert (q[:, :3] == 0).all() and (q[:, 4] == 0).all()
