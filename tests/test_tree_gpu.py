"""Attention of drafted tokens over a paged cache (fa_fwd_tree) against the float64
definition, sequence by sequence and head by head.

Tolerances: the repository's bf16 bounds for O (rel-L2 5e-3, max-abs 2e-2 or four bf16
half-steps of the largest value: P is rounded once, O once; the pieces are joined in
float32), 1e-4 for the float32 LSE.
"""
import numpy as np
import pytest
import torch

import mod_reference as ref
from exact_io_aware_64_b200 import binding
from parity import assert_bf16_close_scaled, to64

pytestmark = pytest.mark.gpu

LSE_ABS = 1e-4


def tree(rng, n, T):
    """[T] ancestor masks as Python ints: token t hangs below an earlier one, or none."""
    bits = []
    for t in range(T):
        parent = int(rng.integers(-1, t)) if t else -1
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << t)
    return bits


def signed(x):
    return x - (1 << 64) if x >> 63 else x


def build(B, H, Hkv, T, lens, d, page, seed, spare=2, poison=True):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + spare
    K = (torch.randn(total, Hkv, page, d, generator=g) * 1.5).bfloat16()
    V = torch.randn(total, Hkv, page, d, generator=g).bfloat16()
    Q = (torch.randn(B, H, T, d, generator=g) * 1.5).bfloat16()
    ids = rng.permutation(total)
    width = max(pages + [1]) + 1
    table = np.full((B, width), 1 << 30, dtype=np.int32)  # entries that are not read
    at = 0
    used = torch.zeros(total, page, dtype=torch.bool)
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        for j in range(lens[b]):
            used[table[b, j // page], j % page] = True
        at += n
    if poison:  # whatever lies behind a sequence's end, or in no sequence
        bad = torch.where(torch.rand(total, 1, page, 1, generator=g) < 0.5, float("nan"),
                          float("inf")).bfloat16()
        K = torch.where(used[:, None, :, None], K, bad)
        V = torch.where(used[:, None, :, None], V, bad)
    return Q, K, V, torch.from_numpy(table)


def check(B, H, Hkv, T, lens, d, page, *, drafted=None, mask=True, softcap=0.0, seed=0,
          heads=None):
    Q, K, V, table = build(B, H, Hkv, T, lens, d, page, seed)
    rng = np.random.default_rng(seed + 1)
    drafted_ = [T] * B if drafted is None else drafted
    bits = [tree(rng, n, T) for n in drafted_]
    tm = torch.tensor([[signed(x) for x in r] for r in bits], dtype=torch.int64) if mask else None
    O = torch.full((B, H, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, H, T), 7.0, device="cuda")
    binding.fwd_tree(Q.cuda(), K.cuda(), V.cuda(), table.cuda(),
                     torch.tensor(lens, dtype=torch.int32).cuda(),
                     seqlens_q=None if drafted is None else
                     torch.tensor(drafted, dtype=torch.int32).cuda(),
                     tree_mask=None if tm is None else tm.cuda(), softcap=softcap, O=O, LSE=LSE)
    binding.check_device_error()
    scale = d ** -0.5
    for b in range(B):
        n, L = drafted_[b], lens[b]
        assert (O[b, :, n:] == 7.0).all() and (LSE[b, :, n:] == 7.0).all()
        if n == 0:
            continue
        j = np.arange(L)
        seen = np.ones((n, L), dtype=bool)
        for t in range(n):
            for u in range(n):
                seen[t, L - n + u] = bool(bits[b][t] >> u & 1) if mask else u <= t
        pg = table[b].numpy()[j // page]
        for h in (range(H) if heads is None else heads):
            c = h // (H // Hkv)
            Kh, Vh = to64(K[pg, c, j % page]), to64(V[pg, c, j % page])
            rO, rL, _ = ref.forward(to64(Q[b, h, :n]), Kh, Vh, scale, seen, softcap)
            assert_bf16_close_scaled(to64(O[b, h, :n]), rO, f"O b={b} h={h}")
            gL = to64(LSE[b, h, :n])
            none = ~seen.any(axis=1)
            assert np.isneginf(gL[none]).all() and (to64(O[b, h, :n])[none] == 0).all()
            assert np.abs(gL[~none] - rL[~none]).max(initial=0.0) <= LSE_ABS


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 384])
@pytest.mark.parametrize("L", [1, 7, 64, 127, 128, 129, 1000])
def test_one_token(L, page, d):
    check(1, 2, 2, 1, [L], d, page, mask=False, seed=L + page)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,T", [(1, 1, 1), (4, 1, 1), (8, 2, 3), (2, 2, 64), (8, 4, 64),
                                     (8, 2, 33), (12, 4, 43), (16, 2, 32), (16, 1, 64), (4, 1, 65 - 1)])
def test_rows(H, Hkv, T, d):
    """Row counts of a key head below, at and above one and two 128-row tiles."""
    check(2, H, Hkv, T, [T + 300, T], d, 16, seed=H + T)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,T", [(4, 2, 1), (4, 2, 17), (8, 2, 60)])
def test_ragged_batch(H, Hkv, T, d):
    """Lengths from nothing to long, sequences with fewer (or no) drafted tokens, more
    sequences than one warp's scan covers."""
    rng = np.random.default_rng(T)
    B = 70
    lens = [int(x) for x in rng.integers(1, 400, B)]
    lens[3], lens[5], lens[6] = 0, T, 2500
    drafted = [int(min(L, rng.integers(0, T + 1))) for L in lens]
    drafted[5] = T
    check(B, H, Hkv, T, lens, d, 32, drafted=drafted, seed=T + d, heads=(0, H - 1))


@pytest.mark.parametrize("T", [1, 16, 64])
def test_chain_is_the_causal_chunk(T):
    """Without a mask the drafted tokens see one another causally: fa_fwd_qk's definition."""
    check(2, 4, 4, T, [T + 131, T + 64], 128, 64, mask=False, seed=T)


@pytest.mark.parametrize("softcap", [0.5, 20.0, 1e5])
@pytest.mark.parametrize("d", [64, 128])
def test_softcap(softcap, d):
    check(2, 8, 2, 5, [700, 90], d, 16, softcap=softcap, seed=11)


def test_long_sequence_split_over_the_gpu():
    check(1, 2, 1, 1, [60000], 128, 64, mask=False, seed=12)
    check(2, 16, 2, 32, [20000, 300], 128, 128, seed=13, heads=(0, 7, 15))


def test_long_tables_of_every_page_size():
    """Tables longer than the 64 entries that the loading warp holds at once."""
    for page in (8, 16, 64, 128, 384):
        check(1, 2, 1, 3, [9000 + page], 64, page, seed=page)


def test_cache_past_32_bits():
    """Pages that begin more than 2^32 bytes (and 2^31 elements) into the cache."""
    page, Hkv, d, L = 64, 8, 128, 500
    num = (1 << 31) // (Hkv * page * d) + 40
    K, V = (torch.empty(num, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    n = -(-L // page)
    ids = torch.arange(num - n, num, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for c in (K, V):
        c[num - n:] = torch.randn(n, Hkv, page, d, generator=g, device="cuda").bfloat16()
    q = torch.randn(1, 16, 1, d, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    O, LSE = binding.fwd_tree(q, K, V, ids[None].contiguous(), lens)
    small = [c[num - n:].clone() for c in (K, V)]
    want, wl = binding.fwd_tree(q, *small, (ids - (num - n))[None].contiguous(), lens)
    binding.check_device_error()
    assert torch.equal(O, want) and torch.equal(LSE, wl)


def test_outputs_made_on_a_given_stream():
    """With fewer drafted tokens than rows and no outputs given, the rows behind them are
    zeros and -inf, filled on the stream that the kernels run on."""
    Q, K, V, table = build(3, 4, 2, 8, [90, 60, 8], 128, 16, 21)
    args = (Q.cuda(), K.cuda(), V.cuda(), table.cuda(),
            torch.tensor([90, 60, 8], dtype=torch.int32).cuda())
    n = torch.tensor([8, 0, 3], dtype=torch.int32).cuda()
    want, wl = binding.fwd_tree(*args, seqlens_q=n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        O, L = binding.fwd_tree(*args, seqlens_q=n, stream=side)
    side.synchronize()
    binding.check_device_error()
    assert torch.equal(O, want) and torch.equal(L, wl)
    assert not O[1].any() and not O[2, :, 3:].any()
    assert torch.isneginf(L[1]).all() and torch.isneginf(L[2, :, 3:]).all()
    assert torch.isfinite(L[0]).all() and torch.isfinite(L[2, :, :3]).all()


def test_rows_that_see_nothing():
    """A sequence that is all draft, and masks with no bit: O = 0, LSE = -inf."""
    Q, K, V, table = build(1, 2, 1, 4, [4], 64, 16, 5)
    mask = torch.tensor([[0, 0b0011, 0, 0b1000]], dtype=torch.int64)
    O, LSE = binding.fwd_tree(Q.cuda(), K.cuda(), V.cuda(), table.cuda(),
                              torch.tensor([4], dtype=torch.int32).cuda(), tree_mask=mask.cuda())
    binding.check_device_error()
    assert (O[:, :, [0, 2]] == 0).all() and torch.isneginf(LSE[:, :, [0, 2]]).all()
    p = table[0, 0]
    assert torch.equal(O[0, :, 3].cpu(), V[p, 0, 3][None].expand(2, -1))


def test_lengths_and_pages_out_of_range():
    """A sequence out of range is skipped and reported; the others are computed.  A page
    outside the cache is reported too (its sequence's outputs are then unspecified)."""
    Q, K, V, table = build(3, 2, 1, 2, [40, 40, 40], 64, 16, 6, poison=False)
    good = torch.tensor([40, 40, 40], dtype=torch.int32).cuda()
    args = (Q.cuda(), K.cuda(), V.cuda())
    want, _ = binding.fwd_tree(*args, table.cuda(), good)
    for lens in ([40, -1, 40], [40, 10 ** 6, 40], [40, 1, 40]):
        O = torch.full_like(want, 7.0)
        binding.fwd_tree(*args, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), O=O)
        with pytest.raises(binding.FAError) as e:
            binding.check_device_error()
        assert e.value.status == binding.FA_ERR_INVALID_ARG
        assert (O[1] == 7.0).all() and torch.equal(O[[0, 2]], want[[0, 2]])
    for bad in (-1, K.shape[0], 1 << 30):
        t = table.clone()
        t[1, 1] = bad
        O, _ = binding.fwd_tree(*args, t.cuda(), good)
        with pytest.raises(binding.FAError, match="page"):
            binding.check_device_error()
        assert torch.equal(O[[0, 2]], want[[0, 2]])
    binding.check_device_error()


def test_in_a_cuda_graph_and_on_another_stream():
    """The lengths are read when the kernels run: a captured call follows the cache as it
    grows.  Two graphs that share a workspace give the same bits one after the other."""
    B, H, Hkv, T, d, page = 2, 8, 2, 1, 128, 16
    Q, K, V, table = build(B, H, Hkv, T, [500, 400], d, page, 8, poison=False)
    q, k, v, tb = Q.cuda(), K.cuda(), V.cuda(), table.cuda()
    lens = torch.tensor([300, 200], dtype=torch.int32).cuda()
    ws = torch.empty(binding.tree_workspace_bytes(B, H, Hkv, T, d), dtype=torch.uint8, device="cuda")
    O, LSE = torch.empty_like(q), torch.empty((B, H, T), device="cuda")
    O2 = torch.empty_like(q)
    binding.fwd_tree(q, k, v, tb, lens, O=O, LSE=LSE, workspace=ws)
    graphs = []
    for out in (O, O2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            binding.fwd_tree(q, k, v, tb, lens, O=out, LSE=LSE, workspace=ws)
        graphs.append(g)
    side = torch.cuda.Stream()
    for n in ([300, 200], [500, 1], [128, 400]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for g in graphs:
            g.replay()
        want, wl = binding.fwd_tree(q, k, v, tb, lens)
        side.wait_stream(torch.cuda.current_stream())
        there, _ = binding.fwd_tree(q, k, v, tb, lens, O=torch.empty_like(q), workspace=ws.clone(),
                                    stream=side)
        torch.cuda.synchronize()
        assert torch.equal(O, want) and torch.equal(O2, want) and torch.equal(there, want)
        assert torch.equal(LSE, wl)
    binding.check_device_error()
    del graphs


def test_a_serving_step_with_rotary_and_the_prompt():
    """The operators together, as they are used: a prompt's keys are turned and attended
    with capped scores, they go into the cache, and drafted tokens at the next positions
    attend to them: a chain of drafts gives what the prompt call gives for the whole."""
    B, H, Hkv, N, T, d, page, cap = 1, 4, 2, 200, 6, 64, 16, 30.0
    g = torch.Generator().manual_seed(3)
    q = torch.randn(B, H, N + T, d, generator=g).bfloat16().cuda()
    k = torch.randn(B, Hkv, N + T, d, generator=g).bfloat16().cuda()
    v = torch.randn(B, Hkv, N + T, d, generator=g).bfloat16().cuda()
    f, m = binding.rotary_frequencies(d, factor=4.0, scaling="parts")
    rq, rk = binding.rotary(q, k, f, mscale=m)
    whole, wl = binding.fwd_mod(rq, rk, v, causal=True, softcap=cap)
    dq, dk = binding.rotary(q[:, :, N:], k[:, :, N:], f, first=N, mscale=m)
    assert torch.equal(dq, rq[:, :, N:]) and torch.equal(dk, rk[:, :, N:])
    pages = -(-(N + T) // page)
    kc, vc = (torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for x, c in ((rk, kc), (v, vc)):
        pad = torch.zeros(B, Hkv, pages * page, d, dtype=torch.bfloat16, device="cuda")
        pad[:, :, :N + T] = x
        c.copy_(pad[0].view(Hkv, pages, page, d).transpose(0, 1))
    O, L = binding.fwd_tree(dq.contiguous(), kc, vc,
                            torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous(),
                            torch.tensor([N + T], dtype=torch.int32, device="cuda"), softcap=cap)
    binding.check_device_error()
    assert_bf16_close_scaled(to64(O), to64(whole[:, :, N:]), "drafts against the prompt call")
    assert (L - wl[:, :, N:]).abs().max() <= 2 * LSE_ABS
