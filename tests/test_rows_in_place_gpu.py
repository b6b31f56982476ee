"""Queries and keys turned in place on a fused projection's output, and gradients turned back into one
tensor: the same bits as into tensors of their own, and nothing else is touched."""
import numpy as np
import pytest

from tests.test_rotary_gpu import _gpu, ints  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(2, 4, 2, 33, 128), (1, 3, 1, 1, 64), (3, 8, 8, 5, 64), (2, 5, 2, 70, 256)]


def parts(wide, H, Hk):
    """Views [B, heads, n, d] (packed: [heads, n, d]) of q, k, v in [.., n, H + 2 Hk, d]."""
    x = wide.transpose(-3, -2)
    return x.split((H, Hk, Hk), -3)


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("packed", [False, True], ids=["batch", "packed"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_fused_projection(shape, packed, inter):
    import torch

    import flash_attention_gb300 as fa

    B, H, Hk, n, d = shape
    g = torch.Generator(device="cuda").manual_seed(n)
    lead = (B * n,) if packed else (B, n)
    wide = torch.randn(*lead, H + 2 * Hk, d, generator=g, device="cuda").bfloat16()
    f, _ = fa.rotary_inv_freq(d // 2)
    kw = dict(interleaved=inter, offset=7)
    if packed:
        kw["cu_seqlens"] = ints(np.arange(B + 1) * n)
    q, k, v = parts(wide, H, Hk)
    want = fa.rotary_fwd(q, k, f, **kw)
    back = fa.rotary_bwd(q, k, f, **kw)
    old_v = v.clone()
    x = wide.clone()
    xq, xk, _ = parts(x, H, Hk)
    got = fa.rotary_fwd(xq, xk, f, out=(xq, xk), **kw)
    assert got[0] is xq and got[1] is xk
    xq, xk, xv = parts(x, H, Hk)
    assert torch.equal(xq, want[0]) and torch.equal(xk, want[1]) and torch.equal(xv, old_v)
    # gradients of their own, contiguous, into one tensor
    y = torch.full_like(wide, 7.0)
    yq, yk, yv = parts(y, H, Hk)
    fa.rotary_bwd(q.contiguous(), k.contiguous(), f, out=(yq, yk), **kw)
    assert torch.equal(yq, back[0]) and torch.equal(yk, back[1]) and (yv == 7).all()
    # and in place; k into v's place
    z = wide.clone()
    zq, zk, zv = parts(z, H, Hk)
    fa.rotary_bwd(zq, zk, f, out=(zq, zv), **kw)
    assert torch.equal(zq, back[0]) and torch.equal(zk, k) and torch.equal(zv, back[1])
    assert fa.fa_device_status(True) == fa.FA_OK


def test_rows_on_one_another_are_refused():
    import torch

    import flash_attention_gb300 as fa

    wide = torch.zeros(2, 6, 8, 64, dtype=torch.bfloat16, device="cuda")
    q, k, v = parts(wide, 4, 2)
    f, _ = fa.rotary_inv_freq(64)
    x = wide.transpose(1, 2)
    for out in ((x[:, 1:5], k), (q, x[:, 3:5]), (x[:, 2:6], x[:, 0:2]), (q, x[:, 5:7])):
        with pytest.raises(fa.FaError):
            fa.rotary_fwd(q, k, f, out=out)
    assert (wide == 0).all()
