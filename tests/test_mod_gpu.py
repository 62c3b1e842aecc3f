"""Modified-score attention (fa_fwd_mod, fa_bwd_mod, fa_doc_ranges) against the float64
definition, head by head.

Tolerances.  bf16: the repository's stated bounds (rel-L2 5e-3, max-abs 2e-2 or four bf16
half-steps of the largest value).  They hold for O at any shape: P and O are rounded once
each (2^-9 of the value on average well below the half-step 2^-8).  D is formed from the
rounded O, which leaves up to 2^-8 |O||dO| in every dS however small dS itself is; where
rows see few keys, the gradient is therefore compared with the formula's from the handed
over O as well as, within the max-abs bound and what the rounding of O alone costs
(computed in float64), with the exact one.  LSE is float32.
"""
import itertools

import numpy as np
import pytest
import torch

import mod_reference as ref
from exact_io_aware_64_b200 import binding, inputs
from parity import bf16_max_abs_bound, assert_bf16_close_scaled, errors, to64

pytestmark = pytest.mark.gpu

LSE_ABS = 1e-4


def make(B, H, Hkv, Nq, Nk, d, seed, sigma=1.5):
    a = inputs.make_inputs(B, H, Nq, d, seed=seed, sigma_qk=sigma, with_dO=True)
    b = inputs.make_inputs(B, Hkv, Nk, d, seed=seed + 1, sigma_qk=sigma)
    return {"Q": a["Q"], "dO": a["dO"], "K": b["K"], "V": b["V"]}


def doc_ids(B, N, mean, seed, padding=0):
    rng = np.random.default_rng(seed)
    out = np.full((B, N), -1, dtype=np.int32)
    for b in range(B):
        at, n, end = 0, 0, N - padding * (b + 1) if padding else N
        while at < end:
            k = int(min(end - at, rng.integers(1, 2 * mean)))
            out[b, at:at + k] = n % 3  # ids repeat: only neighbours belong together
            at, n = at + k, n + 1
    return torch.from_numpy(out)


def check(B, H, Hkv, Nq, Nk, d, *, causal=False, softcap=0.0, slopes=None, prefix=None,
          ids=None, seed=1, sigma=1.5, backward=True, exact=True):
    ins = make(B, H, Hkv, Nq, Nk, d, seed, sigma)
    scale = d ** -0.5
    q, k, v, do = (ins[n].cuda() for n in ("Q", "K", "V", "dO"))
    kw = {"causal": causal, "softcap": softcap,
          "slopes": None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda(),
          "prefix": None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
          "docs": None if ids is None else binding.doc_ranges(ids.cuda())}
    O = torch.full_like(q, float("nan"))
    LSE = torch.full((B, H, Nq), float("nan"), device="cuda")
    binding.fwd_mod(q, k, v, O=O, LSE=LSE, **kw)
    binding.check_device_error()
    if backward:
        grads = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        binding.bwd_mod(q, k, v, O, do, LSE, dQ=grads[0], dK=grads[1], dV=grads[2], **kw)
        binding.check_device_error()
    for b in range(B):
        seen = ref.visible(Nq, Nk, causal, None if prefix is None else prefix[b],
                           None if ids is None else ids[b].numpy())
        dk = {n: [0.0, 0.0] for n in range(Hkv)}
        dv = {n: 0.0 for n in range(Hkv)}
        for h in range(H):
            c = h // (H // Hkv)
            Qh, Kh, Vh, Gh = (to64(t) for t in (ins["Q"][b, h], ins["K"][b, c], ins["V"][b, c],
                                                ins["dO"][b, h]))
            sl = None if slopes is None else float(np.float32(slopes[h]))
            rO, rL, _ = ref.forward(Qh, Kh, Vh, scale, seen, softcap, sl)
            gO, gL = to64(O[b, h]), to64(LSE[b, h])
            empty = ~seen.any(axis=1)
            assert (gO[empty] == 0).all() and np.isneginf(gL[empty]).all()
            assert np.isfinite(gL[~empty]).all()
            assert_bf16_close_scaled(gO, rO, f"O b={b} h={h}")
            if (~empty).any():
                err = np.abs(gL[~empty] - rL[~empty]).max()
                assert err <= LSE_ABS, f"LSE b={b} h={h}: {err:.3e}"
            if not backward:
                continue
            given = ref.backward(Qh, Kh, Vh, Gh, scale, seen, softcap, sl, O=gO)
            full = ref.backward(Qh, Kh, Vh, Gh, scale, seen, softcap, sl)
            g = to64(grads[0][b, h])
            assert (g[empty] == 0).all()
            assert_bf16_close_scaled(g, given[0], f"dQ b={b} h={h}")
            max_abs, rel = errors(g, full[0])
            # |dQ - exact| <= |dQ - given| + |given - exact|: the first is held to the bf16
            # bound above, the second is what the rounded O alone costs, in float64
            allowed = bf16_max_abs_bound(full[0]) + np.abs(given[0] - full[0]).max()
            assert max_abs <= allowed, f"dQ exact {max_abs:.3e} > {allowed:.3e}"
            if exact:
                assert rel <= 5e-3, f"dQ b={b} h={h} vs exact: {rel:.3e}"
            dk[c][0] = dk[c][0] + given[1]
            dk[c][1] = dk[c][1] + full[1]
            dv[c] = dv[c] + given[2]
        if backward:
            blind = ~seen.any(axis=0)
            for c in range(Hkv):
                gk, gv = to64(grads[1][b, c]), to64(grads[2][b, c])
                assert (gk[blind] == 0).all() and (gv[blind] == 0).all()
                assert_bf16_close_scaled(gk, dk[c][0], f"dK b={b} head {c}")
                assert_bf16_close_scaled(gv, dv[c], f"dV b={b} head {c}")
                if exact:
                    _, rel = errors(gk, dk[c][1])
                    assert rel <= 5e-3, f"dK b={b} head {c} vs exact: {rel:.3e}"


# ------------------------------------------------------------------ document ranges
@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 1000, 8191, 8192, 8193, 30011])
def test_doc_ranges(N):
    rng = np.random.default_rng(N)
    rows = [np.repeat(np.arange(N), rng.integers(1, 40, N))[:N], np.zeros(N), np.full(N, -1),
            np.arange(N), rng.integers(-2, 2, N)]
    ids = torch.from_numpy(np.stack(rows).astype(np.int32)).cuda()
    starts, ends = binding.doc_ranges(ids)
    for row, s, e in zip(ids.cpu().numpy(), starts.cpu().numpy(), ends.cpu().numpy()):
        row = np.maximum(row, -1)
        edge = np.flatnonzero(np.concatenate([[True], row[1:] != row[:-1]]))
        n = np.diff(np.concatenate([edge, [N]]))
        rs, re = np.repeat(edge, n), np.repeat(edge + n, n)
        j = np.arange(N)
        assert (s == np.where(row < 0, j, rs)).all() and (e == np.where(row < 0, j, re)).all()


# ------------------------------------------------------------------ one modification each
SHAPES = [(1, 1), (1, 5), (100, 100), (127, 129), (128, 128), (129, 129), (200, 333),
          (256, 256), (257, 1000), (600, 600)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq,Nk", SHAPES)
def test_softcap(Nq, Nk, d, causal):
    check(1, 2, 2, Nq, Nk, d, causal=causal, softcap=5.0, seed=Nq + Nk, exact=Nq >= 100)


@pytest.mark.parametrize("softcap", [1e-3, 0.5, 20.0, 1000.0, 1e6])
def test_softcap_range(softcap):
    check(1, 2, 1, 300, 300, 64, causal=True, softcap=softcap, seed=3,
          exact=softcap > 0.1)


@pytest.mark.parametrize("softcap", [200.0, 1e4, 1e6, 1e8])
def test_scores_above_a_hundred_under_a_large_cap(softcap):
    """A cap far above the scores changes little and must not cost them their digits."""
    check(1, 1, 1, 300, 300, 64, causal=True, softcap=softcap, seed=12, sigma=6.0, exact=False)


def test_softcap_saturates():
    """Scores far past the cap: every tanh is +-1 and the derivative vanishes."""
    check(1, 1, 1, 200, 200, 64, softcap=2.0, seed=4, sigma=20.0, exact=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq,Nk", SHAPES + [(300, 1)])
def test_slopes(Nq, Nk, d, causal):
    if causal and Nq > Nk:
        pytest.skip("causal needs Nq <= Nk")
    check(1, 4, 4, Nq, Nk, d, causal=causal, slopes=[0.5, 0.03, 0.0, -0.01], seed=Nq * 3 + Nk,
          exact=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", SHAPES)
def test_prefix(Nq, Nk, d):
    check(5, 1, 1, Nq, Nk, d, causal=True, prefix=[0, Nk // 3, Nk, Nk + 7, -5], seed=Nq + 2 * Nk,
          exact=Nq >= 100)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq,Nk", SHAPES)
def test_documents(Nq, Nk, d, causal):
    for mean, padding in ((3, 0), (90, 5), (400, 1)):
        check(2, 1, 1, Nq, Nk, d, causal=causal, ids=doc_ids(2, Nk, mean, Nk + mean, min(padding, Nk // 3)),
              seed=Nq * 5 + Nk, exact=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 3), (8, 2)])
def test_shared_heads(H, Hkv, d):
    check(2, H, Hkv, 333, 333, d, causal=True, seed=H)
    check(1, H, Hkv, 130, 700, d, causal=False, softcap=30.0, seed=H + 1)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,causal,cap,slope,pre,docs", [
    c for c in itertools.product([64, 128], [False, True], [0.0, 20.0], [False, True],
                                 [False, True], [False, True]) if c[1] or not c[4]])
def test_together(d, causal, cap, slope, pre, docs):
    B, H, Hkv, N = 2, 4, 2, 421
    check(B, H, Hkv, N, N, d, causal=causal, softcap=cap,
          slopes=[0.25, 0.06, 0.015, 0.004] if slope else None,
          prefix=[100, 200] if pre else None, ids=doc_ids(B, N, 120, 9, 4) if docs else None,
          seed=17, exact=False)


def test_no_document_at_all():
    """Every token is padding: no row sees a key, no key is seen."""
    check(2, 2, 1, 300, 300, 128, causal=True, ids=torch.full((2, 300), -1, dtype=torch.int32))


def test_long_documents():
    """Units whose first tile lies far into the row, at both head sizes."""
    for d in (64, 128):
        check(1, 2, 2, 3000, 3000, d, causal=True, softcap=50.0, ids=doc_ids(1, 3000, 700, 5, 60),
              seed=8, exact=False)


@pytest.mark.parametrize("d", [64, 128])
def test_unmodified_matches_the_plain_calls(d):
    """Without a modification the calls give what fwd and bwd give, bit for bit."""
    ins = make(2, 3, 3, 500, 777, d, 5)
    q, k, v, do = (ins[n].cuda() for n in ("Q", "K", "V", "dO"))
    for causal in (False, True):
        O, L = binding.fwd(q, k, v, causal=causal)
        O2, L2 = binding.fwd_mod(q, k, v, causal=causal)
        assert torch.equal(O, O2) and torch.equal(L, L2)
        for a, b in zip(binding.bwd(q, k, v, O, do, L, causal=causal),
                        binding.bwd_mod(q, k, v, O, do, L, causal=causal)):
            assert torch.equal(a, b)


def test_keys_without_queries():
    """Nq = 0: no query sees any key, so dK and dV of every key head are zero."""
    q = torch.empty(2, 6, 0, 64, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn(2, 3, 50, 64, device="cuda").bfloat16() for _ in "kv")
    O, L = binding.fwd_mod(q, k, v, causal=True, softcap=10.0)
    assert O.shape == q.shape and L.shape == (2, 6, 0)
    dK, dV = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    dQ, _, _ = binding.bwd_mod(q, k, v, O, q, L, causal=True, softcap=10.0, dK=dK, dV=dV)
    binding.check_device_error()
    assert dQ.shape == q.shape and not dK.any() and not dV.any()


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace and outputs, overlap freely."""
    sets = []
    for seed in (1, 2):
        ins = make(2, 4, 2, 900, 900, 128, seed)
        q, k, v, do = (ins[n].cuda() for n in ("Q", "K", "V", "dO"))
        kw = {"causal": True, "softcap": 20.0, "docs": binding.doc_ranges(doc_ids(2, 900, 200, seed).cuda())}
        O, L = binding.fwd_mod(q, k, v, **kw)
        sets.append((q, k, v, do, kw, [O, L, *binding.bwd_mod(q, k, v, O, do, L, **kw)],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, (q, k, v, do, kw, _, s) in enumerate(sets):
            O, L = binding.fwd_mod(q, k, v, stream=s, **kw)
            got[i] = [O, L, *binding.bwd_mod(q, k, v, O, do, L, stream=s, **kw)]
    torch.cuda.synchronize()
    binding.check_device_error()
    for g, s in zip(got, sets):
        assert all(torch.equal(a, b) for a, b in zip(g, s[5]))


def test_after_other_work_of_the_stream():
    """The kernels may be launched before the stream's earlier work ends; they must not read
    their inputs, or write outputs that it still reads, before it has.  Eager and captured."""
    B, H, N, d = 1, 8, 1500, 128
    ins = make(B, H, H, N, N, d, 9)
    src = [ins[n].cuda() for n in ("Q", "K", "V", "dO")]
    ids = doc_ids(B, N, 300, 2).cuda()
    bufs = [torch.empty_like(t) for t in src]
    idb = torch.empty_like(ids)
    O, L = torch.empty_like(src[0]), torch.empty((B, H, N), device="cuda")
    grads = [torch.empty_like(t) for t in src[:3]]
    keep = [torch.empty_like(t) for t in (O, *grads)]
    ws = torch.empty(binding.workspace_bytes(B, H, N, d), dtype=torch.uint8, device="cuda")
    rng = [torch.empty_like(ids), torch.empty_like(ids)]

    def step():
        for b, s in zip((*bufs, idb), (*src, ids)):
            b.copy_(s)
        docs = binding.doc_ranges(idb, *rng)
        idb.fill_(-1)
        binding.fwd_mod(*bufs[:3], causal=True, docs=docs, O=O, LSE=L)
        binding.bwd_mod(*bufs[:3], O, bufs[3], L, causal=True, docs=docs, dQ=grads[0], dK=grads[1],
                        dV=grads[2], workspace=ws)
        for k, t in zip(keep, (O, *grads)):
            k.copy_(t)
        for t in (*bufs, O, L, *grads, *rng, ws):
            t.fill_(1)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in keep]
    docs = binding.doc_ranges(ids)
    want, wl = binding.fwd_mod(*src[:3], causal=True, docs=docs)
    torch.cuda.synchronize()
    assert torch.equal(first[0], want)
    for a, b in zip(first[1:], binding.bwd_mod(*src[:3], want, src[3], wl, causal=True, docs=docs)):
        assert torch.equal(a, b)
    for _ in range(20):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, keep))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        step()
    for t in keep:
        t.zero_()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, keep))
    del g


def test_in_a_cuda_graph_and_on_another_stream():
    B, H, Hkv, N, d = 1, 4, 2, 700, 64
    ins = make(B, H, Hkv, N, N, d, 6)
    q, k, v, do = (ins[n].cuda() for n in ("Q", "K", "V", "dO"))
    ids = doc_ids(B, N, 150, 3, 4).cuda()
    starts, ends = torch.empty_like(ids), torch.empty_like(ids)
    outs = [torch.empty_like(q), torch.empty((B, H, N), device="cuda"), torch.empty_like(q),
            torch.empty_like(k), torch.empty_like(v)]
    ws = torch.empty(binding.workspace_bytes(B, H, N, d), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        docs = binding.doc_ranges(ids, starts, ends, stream=stream)
        kw = {"causal": True, "softcap": 10.0, "docs": docs, "stream": stream}
        binding.fwd_mod(q, k, v, O=outs[0], LSE=outs[1], **kw)
        binding.bwd_mod(q, k, v, outs[0], do, outs[1], dQ=outs[2], dK=outs[3], dV=outs[4],
                        workspace=ws, **kw)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    for t in outs:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    binding.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    del g
