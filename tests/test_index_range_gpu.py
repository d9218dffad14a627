"""The index rows at the ends of their values' range."""
import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import serving_ref as R
from tests.test_rope_gpu import check_codes, freqs, split_fused

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


@pytest.mark.parametrize("largest", [2.0 ** 125, 2.0 ** 126, 8.6e37, 1.5e38, 2.0 ** 127, torch.finfo(torch.bfloat16).max])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, True), (128, False)])
def test_rows_of_large_finite_values(largest, rot, interleaved):
    """A row's largest magnitude becomes 448 up to the end of the type.  A
    token at position 0 turns by nothing, so that no rotated value passes
    fp32."""
    g = R.gen(rot)
    n, heads = 5, 3
    q = torch.rand((n, heads, 128), generator=g) * 2 - 1
    k = torch.rand((n, 128), generator=g) * 2 - 1
    q[..., 17], k[..., 101] = 1.0, -1.0
    q[2, 1] = 1.0
    q, k = ((x * largest).bfloat16() for x in (q, k))
    assert torch.isfinite(q).all() and q.abs().amax() == torch.tensor(largest).bfloat16()
    w = torch.ones((n, heads))
    pos, req = torch.zeros(n, dtype=torch.int32), torch.arange(n, dtype=torch.int32)
    table = torch.tensor([[4], [2], [0], [1], [3]], dtype=torch.int32)
    kv = torch.zeros((n, 8448), dtype=torch.uint8, device="cuda")
    f = freqs(rot)
    qo, wo = pml.pml_index_quant_append(q.cuda(), k.cuda(), w.cuda(), pos.cuda(), req.cuda(), f.cuda(), kv,
                                        table.cuda(), interleaved=interleaved)
    assert pml.pml_device_status(clear=True) == 0
    want, size = R.rope(q, pos, f, 0, interleaved)
    codes = qo.cpu().double()
    assert (codes.abs().amax(-1) == 448).all()
    check_codes(codes, wo.cpu().double(), want, size)
    want, size = R.rope(k[:, None], pos, f, 0, interleaved)
    keys, scales = split_fused(kv)
    page = table[:, 0].long()
    assert (keys[page, 0].abs().amax(-1) == 448).all()
    check_codes(keys[page, 0], scales[page, 0], want[:, 0], size[:, 0])


def test_small_rows_keep_their_codes():
    """Rows around the least scale, 1e-12 / 448, and far below it."""
    x = torch.ones((4, 1, 128)) * torch.tensor([1e-11, 1e-12, 1e-13, 1e-38])[:, None, None]
    q = x.bfloat16()
    qo, wo = pml.pml_index_quant_append(q.cuda(), None, torch.ones((4, 1)).cuda(), torch.arange(4).cuda(), None,
                                        freqs(0).cuda(), None, None)
    check_codes(qo.cpu().double(), wo.cpu().double(), q.double(), q.double().abs())


@pytest.mark.parametrize("keys", [False, True])
def test_padding_tokens(keys):
    """Nothing of a token with a negative position (or, with keys, request) is
    written."""
    g = R.gen(5)
    n, heads = 40, 5
    q, k = torch.randn((n, heads, 128), generator=g).bfloat16(), torch.randn((n, 128), generator=g).bfloat16()
    pos = torch.arange(n)
    pos[[0, 7, 39]] = torch.tensor([-1, -2 ** 40, -64])
    req = torch.zeros(n, dtype=torch.int32)
    real = pos >= 0
    if keys:
        req[3], real[3] = -1, False
    kv = torch.full((1, 8448), 9, dtype=torch.uint8, device="cuda")
    qo = torch.full((n, heads, 128), 7, dtype=torch.uint8, device="cuda")
    wo = torch.full((n, heads), 5.0, device="cuda")
    w = torch.ones((n, heads)).cuda()
    more = (k.cuda(), req.cuda(), kv, torch.zeros((1, 1), dtype=torch.int32, device="cuda")) if keys else (None,) * 4
    pml.pml_index_quant_append(q.cuda(), more[0], w, pos.cuda(), more[1], freqs(64).cuda(), more[2], more[3], qo, wo)
    assert pml.pml_device_status(clear=True) == 0
    want, size = R.rope(q, pos, freqs(64))
    codes = qo.cpu().view(torch.float8_e4m3fn).double()
    check_codes(codes[real], wo.cpu().double()[real], want[real], size[real])
    assert (qo.cpu()[~real] == 7).all() and (wo.cpu()[~real] == 5.0).all()
    assert ((kv[0, :8192].reshape(64, 128) != 9).any(1).sum() == real.sum()) if keys else (kv == 9).all()
