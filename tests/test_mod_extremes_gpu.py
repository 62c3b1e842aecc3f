"""Modified-score attention (fa_fwd_mod, fa_bwd_mod) where hidden and visible scores lie far
apart, against the float64 definition, head by head.

Tolerances, element by element, half a step of bf16 being 2^-8 of a value.  A float32 score x
is off by 1.1e-6 |x| where the cap is the polynomial, by 2^-22 cap where it is the formula
(below 4.3e-5 for caps up to 177, which use it for whole tiles; below 2^-19 |x| for larger
ones, which use it above a fifth of the cap), and by 2^-21 |x| for the product, the scale, the
subtraction of the maximum and the logarithm: by 2^-19 |x| + 4.3e-5.  LSE may be off by 2^-19
|x| + 1e-4, a probability by
  eP = P (2^-8 + 2^-18 |x| + 1e-4)
(its rounding, its score and LSE or sum, the exponential), dP - D by 2^-20 of the products that
make it (d and Nk of them in float32, whose roundings add up like their root), and
  eS = |dS| (2^-8 + 2^-18 |x| + 3e-4) + P dz 2^-20 (|dO| |V|^T + |dO| . |O|)
(3e-4: the cap's derivative, 1.6e-4, beside eP's; and P |dP - D| 2^-21 where that is 1 - tanh^2
of a float32 tanh, off by 2^-23 at 1, squared, subtracted).  Then O, dV, dQ and dK are off by
eP |V|, eP^T |dO|, scale eS |K| and scale eS^T |Q| and by their own rounding.  These bounds do
not presume scores of any size: where all of a row's keys share a large column, its dQ there
is a difference of large products, each rounded.  The gradients are compared with the
formula's from the O that the call is handed.
"""
import numpy as np
import pytest
import torch

import mod_reference as ref
from exact_io_aware_64_b200 import binding
from parity import to64

pytestmark = pytest.mark.gpu


HALF = 2.0 ** -8


def assert_within(got, want, bound, what):
    # (1e-12: the float64 sums themselves, and 1 - tanh^2 of saturated scores in them)
    over = np.abs(got - want) - (bound + HALF * np.abs(want) + 1e-12)
    assert over.max(initial=0.0) <= 0, f"{what}: {over.max():.3e} over its bound"


def check(q, k, v, do, *, causal=False, softcap=0.0, slopes=None, prefix=None, ids=None,
          heads=None, sequences=None):
    """Forward and backward of bf16 CPU tensors against float64, for the given query heads'
    O, LSE and dQ and, where all the heads of a key head are given, its dK and dV."""
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    scale = d ** -0.5
    kw = {"causal": causal, "softcap": softcap,
          "slopes": None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda(),
          "prefix": None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
          "docs": None if ids is None else binding.doc_ranges(ids.cuda())}
    gpu = [t.cuda() for t in (q, k, v)]
    O = torch.full_like(gpu[0], float("nan"))
    LSE = torch.full((B, H, Nq), float("nan"), device="cuda")
    binding.fwd_mod(*gpu, O=O, LSE=LSE, **kw)
    grads = [torch.full_like(t, float("nan")) for t in gpu]
    binding.bwd_mod(*gpu, O, do.cuda(), LSE, dQ=grads[0], dK=grads[1], dV=grads[2], **kw)
    binding.check_device_error()
    assert all(torch.isfinite(t).all() for t in (O, *grads))
    heads = range(H) if heads is None else heads
    for b in range(B) if sequences is None else sequences:
        seen = ref.visible(Nq, Nk, causal, None if prefix is None else prefix[b],
                           None if ids is None else ids[b].numpy())
        empty, blind = ~seen.any(axis=1), ~seen.any(axis=0)
        sums, n = {}, {}
        for h in heads:
            c = h // (H // Hkv)
            Qh, Kh, Vh, Gh = (to64(t) for t in (q[b, h], k[b, c], v[b, c], do[b, h]))
            sl = None if slopes is None else float(np.float32(slopes[h]))
            rO, rL, P = ref.forward(Qh, Kh, Vh, scale, seen, softcap, sl)
            x, dz = ref.scores(Qh, Kh, scale, softcap, sl)
            gO, gL = to64(O[b, h]), to64(LSE[b, h])
            assert (gO[empty] == 0).all() and np.isneginf(gL[empty]).all()
            ax = np.where(seen, np.abs(x), 0.0).max(axis=1, keepdims=True)
            off = np.abs(gL[~empty] - rL[~empty]) - (1e-4 + 2.0 ** -19 * ax[~empty, 0])
            assert off.max(initial=0.0) <= 0, f"LSE b={b} h={h}: {off.max():.3e} over its bound"
            eP = P * (HALF + 2.0 ** -18 * ax + 1e-4)
            assert_within(gO, rO, eP @ np.abs(Vh), f"O b={b} h={h}")
            dQ, dK, dV = ref.backward(Qh, Kh, Vh, Gh, scale, seen, softcap, sl, O=gO)
            D = (Gh * gO).sum(axis=1, keepdims=True)
            dP = np.abs(P * (Gh @ Vh.T - D))
            eS = (dP * dz * (HALF + 2.0 ** -18 * ax + 3e-4) + dP * 2.0 ** -21 +
                  P * dz * 2.0 ** -20 * (np.abs(Gh) @ np.abs(Vh).T +
                                         (np.abs(Gh) * np.abs(gO)).sum(axis=1, keepdims=True)))
            g = to64(grads[0][b, h])
            assert (g[empty] == 0).all()
            assert_within(g, dQ, scale * eS @ np.abs(Kh), f"dQ b={b} h={h}")
            mine = (dK, scale * eS.T @ np.abs(Qh), dV, eP.T @ np.abs(Gh))
            sums[c] = [s + t for s, t in zip(sums.get(c, (0.0,) * 4), mine)]
            n[c] = n.get(c, 0) + 1
        for c, (dK, eK, dV, eV) in sums.items():
            gk, gv = to64(grads[1][b, c]), to64(grads[2][b, c])
            assert (gk[blind] == 0).all() and (gv[blind] == 0).all()
            if n[c] == H // Hkv:
                assert_within(gk, dK, eK, f"dK b={b} head {c}")
                assert_within(gv, dV, eV, f"dV b={b} head {c}")


# ------------------------------------------------------------------ scores of given size
def placed(z, Nq, d, seed):
    """Q [1, 1, Nq, d], K [1, 1, Nk, d], V, dO whose scaled scores are z[j] (z: [Nk]) plus
    products of deviation about 0.3: the first column holds z, the others noise."""
    g = torch.Generator().manual_seed(seed)
    Nk = len(z)
    q, do = (torch.randn(1, 1, Nq, d, generator=g) for _ in "qg")
    k, v = (torch.randn(1, 1, Nk, d, generator=g) for _ in "kv")
    q, k = q * 0.5, k * 0.5
    q[..., 0] = 8.0
    k[0, 0, :, 0] = torch.tensor(z) * d ** 0.5 / 8.0
    return [t.bfloat16() for t in (q, k, v, do)]


# (cap, visible scores, hidden ones beside them): visible scores down towards the cap, hidden
# ones on both sides of what a tile takes the polynomial for
FAR = [(cap, low, hid) for cap, low in ((50.0, -90.0), (60.0, -120.0), (100.0, -95.0), (200.0, -120.0),
                                        (1000.0, -300.0), (1e4, -300.0))
       for hid in (0.0, 33.0, -33.0)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap,low,hidden", FAR)
def test_hidden_document_before_low_scores(softcap, low, hidden, d):
    """Rows walk a key tile of another document, whose scores would be the larger ones by
    far, before the tile of their own."""
    ids = torch.tensor([[0] * 128 + [1] * 128 + [2] * 60 + [3] * 84], dtype=torch.int32)
    z = [hidden] * 128 + [low] * 128 + [hidden] * 60 + [low] * 84
    for causal in (False, True):
        check(*placed(z, 400, d, 1), softcap=softcap, ids=ids, causal=causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap,low,hidden", FAR)
def test_hidden_keys_behind_low_scores(softcap, low, hidden, d):
    """The first rows of a row tile do not see its last key tile, whose scores would be the
    larger ones: causal with a position in mid-tile, and keys behind a prefix."""
    z = [low] * 128 + [hidden] * 64
    check(*placed(z, 128, d, 2), softcap=softcap, causal=True)
    z = [low] * 256 + [hidden] * 72
    check(*placed(z, 328, d, 3), softcap=softcap, causal=True, prefix=[130])


@pytest.mark.parametrize("softcap", [60.0, 100.0, 1000.0])
def test_low_and_hidden_scores_in_one_tile(softcap):
    """Visible keys of both sizes among hidden ones, document by document."""
    rng = np.random.default_rng(4)
    N = 700
    ids = np.cumsum(rng.random(N) < 0.03).astype(np.int32)
    z = rng.choice([-1.4 * softcap, -33.0, 0.0, 33.0], size=ids.max() + 1)[ids]
    check(*placed(z.tolist(), N, 64, 5), softcap=softcap, causal=True,
          ids=torch.from_numpy(ids)[None])


# ------------------------------------------------------------------ caps near nothing
@pytest.mark.parametrize("softcap", [1.1e-9, 1e-8, 1e-7, 5e-7, 1e-6, 1e-3])
@pytest.mark.parametrize("d", [64, 128])
def test_zero_queries_under_a_small_cap(softcap, d):
    """Rows whose every product is zero (padding), beside rows that saturate: equal weights."""
    g = torch.Generator().manual_seed(6)
    q, do = (torch.randn(1, 4, 300, d, generator=g).bfloat16() for _ in "qg")
    k, v = (torch.randn(1, 2, 300, d, generator=g).bfloat16() for _ in "kv")
    q[:, :, :100] = 0
    q[:, 1] = 0
    for causal in (False, True):
        check(q, k, v, do, softcap=softcap, causal=causal)
    check(q, k, v, do, softcap=softcap, causal=True, slopes=[0.5, 0.1, 0.0, 0.02])


@pytest.mark.parametrize("softcap", [1.1e-9, 1e-7, 1e-6])
def test_zero_query_under_a_small_cap_over_a_paged_cache(softcap):
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(40, 2, 16, 64, generator=g).bfloat16() for _ in "kv")
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    q[0, 3] = torch.randn(1, 64, generator=g).bfloat16()
    table = torch.arange(40, dtype=torch.int32)[None].contiguous()
    lens = torch.tensor([600], dtype=torch.int32)
    O, LSE = binding.fwd_tree(*(t.cuda() for t in (q, k, v, table, lens)), softcap=softcap)
    binding.check_device_error()
    # every weight is 1 / 600, rounded; so is the output
    flat = to64(v.transpose(0, 1).reshape(2, 640, 64)[:, :600])
    for h in range(4):
        bound = HALF * np.abs(flat[h // 2]).mean(axis=0)[None] * 1.01
        assert_within(to64(O[0, h]), flat[h // 2].mean(axis=0)[None], bound, f"O h={h}")
    assert np.abs(to64(LSE) - np.log(600.0)).max() <= 1e-4


# ------------------------------------------------------------------ many units a CTA
def rows_of_documents(B, N, seed, gaps):
    """Documents of 1 to 500 tokens with runs of padding (first, last) between them."""
    rng = np.random.default_rng(seed)
    ids = np.stack([np.cumsum(rng.random(N) < 0.01) for _ in range(B)]).astype(np.int32)
    for b in range(B):
        for first, last in gaps:
            ids[b, min(N, first + 40 * b):min(N, last + 40 * b)] = -1
    return torch.from_numpy(ids)


def tensors(B, H, Hkv, Nq, Nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    q, do = (torch.randn(B, H, Nq, d, generator=g) for _ in "qg")
    k, v = (torch.randn(B, Hkv, Nk, d, generator=g) for _ in "kv")
    return [t.bfloat16() for t in (q * 1.5, k * 1.5, v, do)]


MODS = [{}, {"softcap": 20.0}, {"slopes": True}, {"softcap": 20.0, "slopes": True}]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mods", MODS, ids=["mask", "cap", "bias", "both"])
def test_several_units_a_block(mods, d):
    """384 forward, 192 dK/dV and 768 dQ units for 148 SMs, ranked by cost; dead units, and
    units with one live row tile, among them."""
    B, H, Hkv, N = 4, 16, 4, 1500
    kw = dict(mods)
    if "slopes" in kw:
        kw["slopes"] = [2.0 ** (-h / 2) for h in range(1, H + 1)]
    ids = rows_of_documents(B, N, 8, [(250, 640), (900, 1300)])
    check(*tensors(B, H, Hkv, N, N, d, 9), ids=ids, causal=True, heads=(4, 5, 6, 7),
          sequences=(0, 3), **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mods", MODS[:2], ids=["mask", "cap"])
def test_queries_in_front_of_the_first_key(mods, d):
    """Nq > Nk with documents: whole units, and the first row tile of one (rows 256 to 383 see
    nothing, those behind them do), lie in front of the first key."""
    B, H, Hkv, Nk = 3, 16, 8, 1100
    check(*tensors(B, H, Hkv, Nk + 384, Nk, d, 10), heads=(2, 3), sequences=(0, 2),
          ids=rows_of_documents(B, Nk, 11, [(300, 700)]), **mods)


@pytest.mark.parametrize("d", [64, 128])
def test_units_too_many_to_be_ranked(d):
    """More than 256 row tile pairs over the batch: dealt in index order."""
    B, N = 70, 1000
    ids = rows_of_documents(B, N, 12, [(100, 500)])
    for causal in (False, True):
        check(*tensors(B, 2, 1, N, N, d, 13), ids=ids, causal=causal, softcap=20.0,
              sequences=(0, 9, 69))


@pytest.mark.parametrize("d", [64, 128])
def test_several_units_without_documents(d):
    check(*tensors(2, 32, 16, 2000, 2000, d, 14), causal=True, softcap=20.0, prefix=[900, 0],
          heads=(0, 1), sequences=(0, 1))
    check(*tensors(3, 16, 4, 900, 1900, d, 15), heads=(12, 13, 14, 15), sequences=(2,))
