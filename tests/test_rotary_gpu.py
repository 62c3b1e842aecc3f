"""Rotary positions (fa_rotary, fa_rotary_f32) against the float64 definition.

Tolerances, from the arithmetic.  The angle reaches float32 as a fraction of a half turn in
[-1, 1], rounded by 2^-25 at most: pi 2^-25 < 1.6 2^-24 rad; float64 leaves 2^-51 of
|position * inv_freq| (two roundings there, two in the test).  sincospi is within 2 float32
steps (2 * 2^-23 = 4 * 2^-24 of at most 1), its product with mscale, the two products with x
and their sum round by 2^-24 each: (1.6 + 4 + 1 + 1 + 1) 2^-24 < 9 2^-24 of m (|x1| + |x2|).
A bf16 output rounds by 2^-8 of the value more.
"""
import numpy as np
import pytest
import torch

from exact_io_aware_64_b200 import binding

pytestmark = pytest.mark.gpu


def expected(x, freq, pos, interleaved, mscale, sign=1.0):
    """x [B, heads, N, d], freq [R/2], pos [B, N] float64 -> (y, bound of y's error)."""
    R = 2 * freq.size
    ang = pos[:, None, :, None] * freq
    a = np.arange(R // 2)
    a, b = (2 * a, 2 * a + 1) if interleaved else (a, a + R // 2)
    c, s = mscale * np.cos(ang), sign * mscale * np.sin(ang)
    y, bound = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size = abs(mscale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    bound[..., a] = bound[..., b] = size * (9 * 2.0 ** -24 + 2.0 ** -51 * np.abs(ang))
    return y, bound


def assert_within(got, y, bound):
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(y)
    got = got.double().cpu().numpy()
    over = np.abs(got - y) - bound
    assert (over <= 0).all(), f"off by {over.max():.3e} more than the bound"


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def freqs(R):
    return binding.rotary_frequencies(R)[0] if R else torch.empty(0, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R", [(64, 64), (128, 128), (128, 64), (64, 16), (128, 124), (64, 2),
                                 (128, 0), (80, 20), (66, 34), (512, 512)])
@pytest.mark.parametrize("B,H,Hkv,N", [(1, 1, 1, 1), (2, 4, 2, 37), (3, 5, 1, 300)])
def test_values(B, H, Hkv, N, d, R, interleaved, dtype):
    q, k = rand((B, H, N, d), dtype, 1), rand((B, Hkv, N, d), dtype, 2)
    f = freqs(R)
    pos = torch.randint(0, 100000, (B, N), generator=torch.Generator().manual_seed(3)).int()
    oq, ok = binding.rotary(q.cuda(), k.cuda(), f, positions=pos.cuda(), interleaved=interleaved,
                            mscale=1.25)
    for x, out in ((q, oq), (k, ok)):
        y, bound = expected(x.double().numpy(), f.double().cpu().numpy(), pos.double().numpy(),
                            interleaved, 1.25)
        assert_within(out, y, bound)
        assert torch.equal(out[..., R:].cpu(), x[..., R:])


@pytest.mark.parametrize("first", [0, 7, 1 << 20, (1 << 31) - 5, -1000])
def test_positions(first):
    """Far, negative and counted positions; int32 positions give the same bits as `first`."""
    x = rand((2, 3, 50, 64), torch.float32, 4)
    f = freqs(64)
    out, _ = binding.rotary(x.cuda(), None, f, first=first)
    pos = first + np.arange(50, dtype=np.float64)[None].repeat(2, 0)
    assert_within(out, *expected(x.double().numpy(), f.double().cpu().numpy(), pos, False, 1.0))
    if abs(first) < (1 << 31) - 100:
        p = torch.from_numpy(pos).int().cuda()
        assert torch.equal(out, binding.rotary(x.cuda(), None, f, positions=p)[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved, dtype):
    """The gradient against the formula, and against differences: the map is linear, so
    <g, f(x + e) - f(x)> = <grad, e> for any e, exactly but for the roundings."""
    B, H, N, d, R = 2, 3, 65, 128, 96
    g = rand((B, H, N, d), dtype, 5)
    f = freqs(R)
    kw = {"first": 1234, "interleaved": interleaved, "mscale": 0.75}
    grad, none = binding.rotary_bwd(g.cuda(), None, f, **kw)
    assert none is None
    pos = 1234 + np.arange(N, dtype=np.float64)[None].repeat(B, 0)
    y, bound = expected(g.double().numpy(), f.double().cpu().numpy(), pos, interleaved, 0.75, -1.0)
    assert_within(grad, y, bound)
    e = rand((B, H, N, d), torch.float32, 6)
    fe, _ = binding.rotary(e.cuda(), None, f, **kw)
    lhs = (g.double() * fe.double().cpu()).sum(-1)
    rhs = (grad.double().cpu() * e.double()).sum(-1)
    # a row's products: every term off by the bounds above (bf16: 2^-8 of grad's elements)
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    allowed = ((20 * 2.0 ** -24 + step) * 2 * (g.double().abs() * 2).norm(dim=-1) *
               (e.double().abs() * 2).norm(dim=-1))
    assert ((lhs - rhs).abs() <= allowed).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layouts(dtype):
    """Slices of a fused projection, in place and not, packed tokens, odd offsets: the bits
    of the contiguous call."""
    B, H, Hkv, N, d = 2, 4, 2, 100, 64
    f = freqs(d)
    pos = torch.arange(B * N).view(B, N).int().cuda() * 3
    fused = rand((B, N, (H + 2 * Hkv), d), dtype, 7).cuda()
    q, k = fused[:, :, :H].transpose(1, 2), fused[:, :, H:H + Hkv].transpose(1, 2)
    oq, ok = binding.rotary(q.contiguous(), k.contiguous(), f, positions=pos)
    sq, sk = binding.rotary(q, k, f, positions=pos)
    assert torch.equal(sq, oq) and torch.equal(sk, ok)
    copy = fused.clone()
    q2, k2 = copy[:, :, :H].transpose(1, 2), copy[:, :, H:H + Hkv].transpose(1, 2)
    binding.rotary(q2, k2, f, positions=pos, Q_out=q2, K_out=k2)
    assert torch.equal(q2, oq) and torch.equal(k2, ok)
    assert torch.equal(copy[:, :, H + Hkv:], fused[:, :, H + Hkv:])
    # packed: the tokens of all sequences one after another
    pq = q.transpose(1, 2).reshape(B * N, H, d).contiguous()
    po, none = binding.rotary(pq, None, f, positions=pos.view(-1))
    assert none is None and torch.equal(po.view(B, N, H, d).transpose(1, 2), oq)
    # one element off a 16-byte boundary
    buf = torch.empty(B * H * N * d + 1, dtype=dtype, device="cuda")[1:].view(B, H, N, d)
    buf.copy_(q)
    off, _ = binding.rotary(buf, None, f, positions=pos)
    assert torch.equal(off, oq)


def test_partial_head_in_place_keeps_the_rest():
    x = rand((1, 2, 33, 128), torch.bfloat16, 8).cuda()
    want, _ = binding.rotary(x, None, freqs(32), first=5)
    y = x.clone()
    binding.rotary(y, None, freqs(32), first=5, Q_out=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("scaling", ["linear", "base", "parts"])
def test_scaled_frequencies(scaling):
    f, m = binding.rotary_frequencies(128, factor=8.0, scaling=scaling, original_len=4096)
    f0, _ = binding.rotary_frequencies(128)
    r = (f0.double() / f.double()).cpu().numpy()
    assert (r > 1 - 1e-6).all() and (r < 8 + 1e-5).all()
    if scaling == "linear":
        assert np.allclose(r, 8.0, rtol=1e-6) and m == 1.0
    else:
        assert abs(r[0] - 1) < 1e-6 and abs(r[-1] - 8) < 1e-5 and (np.diff(r) >= -1e-6).all()
    assert scaling != "parts" or abs(m - (0.1 * np.log(8.0) + 1)) < 1e-12


def test_empty_and_many_heads():
    f = freqs(64)
    for shape in ((0, 4, 10, 64), (2, 4, 0, 64), (2, 0, 10, 64)):
        out, _ = binding.rotary(torch.empty(shape, device="cuda"), None, f)
        assert out.shape == shape
    x = rand((1, 700, 3, 64), torch.bfloat16, 9)
    out, _ = binding.rotary(x.cuda(), None, f, first=11)
    pos = 11 + np.arange(3, dtype=np.float64)[None]
    assert_within(out, *expected(x.double().numpy(), f.double().cpu().numpy(), pos, False, 1.0))


def test_in_a_cuda_graph_and_on_another_stream():
    q, k = rand((2, 4, 77, 64), torch.bfloat16, 1).cuda(), rand((2, 2, 77, 64), torch.bfloat16, 2).cuda()
    f = freqs(64)
    want = [t.clone() for t in binding.rotary(q, k, f, first=3)]
    oq, ok = torch.zeros_like(q), torch.zeros_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.rotary(q, k, f, first=3, Q_out=oq, K_out=ok, stream=side)
    side.synchronize()
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        binding.rotary(q, k, f, first=3, Q_out=oq, K_out=ok)
    oq.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
    del g
