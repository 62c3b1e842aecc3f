"""Rotary positions of a fused projection's slices, handed on to the attention calls as they
come."""
import pytest
import torch

from exact_io_aware_64_b200 import binding

pytestmark = pytest.mark.gpu


def fused(B, N, H, Hkv, d, seed):
    x = torch.randn(B, N, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(seed))
    return x.bfloat16().cuda()


def test_slices_into_modified_scores_and_back():
    """Forward, backward and the positions' gradient give what contiguous copies give."""
    B, N, H, Hkv, d = 2, 150, 4, 2, 64
    x = fused(B, N, H, Hkv, d, 1)
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    v = v.contiguous()
    f, m = binding.rotary_frequencies(d, factor=4.0, scaling="parts")
    want_q, want_k = binding.rotary(q.contiguous(), k.contiguous(), f, mscale=m)
    rq, rk = binding.rotary(q, k, f, mscale=m)
    assert torch.equal(rq, want_q) and torch.equal(rk, want_k)
    kw = {"causal": True, "softcap": 20.0}
    O, L = binding.fwd_mod(rq, rk, v, **kw)
    want, wl = binding.fwd_mod(want_q, want_k, v, **kw)
    assert torch.equal(O, want) and torch.equal(L, wl)
    dO = torch.randn(B, H, N, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    dq, dk, _ = binding.bwd_mod(rq, rk, v, O, dO, L, **kw)
    gq, gk = binding.rotary_bwd(dq, dk, f, mscale=m)
    # gradients go back into the projection's own layout
    dx = torch.zeros_like(x)
    binding.rotary_bwd(dq, dk, f, mscale=m, dQ=dx[:, :, :H].transpose(1, 2),
                       dK=dx[:, :, H:H + Hkv].transpose(1, 2))
    assert torch.equal(dx[:, :, :H].transpose(1, 2), gq)
    assert torch.equal(dx[:, :, H:H + Hkv].transpose(1, 2), gk) and not dx[:, :, H + Hkv:].any()
    binding.check_device_error()


def test_packed_slices_into_the_packed_call():
    T, H, d = 200, 3, 128
    x = torch.randn(T, 3 * H, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q, k, v = (x[:, a:a + H] for a in (0, H, 2 * H))
    f, _ = binding.rotary_frequencies(d)
    rq, rk = binding.rotary(q, k, f, positions=torch.arange(T, dtype=torch.int32, device="cuda"))
    cu = torch.tensor([0, 90, T], dtype=torch.int32, device="cuda")
    O, L = binding.fwd_packed(rq, rk, v.contiguous(), cu, cu, 110, 110, causal=True)
    binding.check_device_error()
    assert torch.isfinite(O).all() and torch.isfinite(L).all()


def test_drafted_slices_into_the_paged_call():
    B, T, H, Hkv, d = 3, 5, 4, 2, 64
    x = fused(B, T, H, Hkv, d, 4)
    f, _ = binding.rotary_frequencies(d)
    q = x[:, :, :H].transpose(1, 2)
    cache = torch.randn(12, Hkv, 16, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(B, 4).contiguous()
    lens = torch.tensor([64, 40, 7], dtype=torch.int32, device="cuda")
    rq, none = binding.rotary(q, None, f, first=35)
    assert none is None
    O, L = binding.fwd_tree(rq, cache, cache, table, lens)
    want, wl = binding.fwd_tree(binding.rotary(q.contiguous(), None, f, first=35)[0], cache, cache,
                                table, lens)
    binding.check_device_error()
    assert torch.equal(O, want) and torch.equal(L, wl)
