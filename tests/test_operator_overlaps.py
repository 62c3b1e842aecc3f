"""Buffers that a call writes and another argument shares: refused on the host (no GPU; an
accepted call gets as far as asking for a device)."""
import ctypes

import numpy as np
import pytest
import torch

from exact_io_aware_64_b200 import binding

BAD = binding.FA_ERR_INVALID_ARG
BASE = 1 << 40
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="its addresses are made up")


def refused(fn, args):
    lib = binding.lib()
    status = getattr(lib, fn)(*args)
    msg = lib.fa_last_error_message().decode()
    assert (status == BAD) == bool("overlap" in msg or "share" in msg or "same output" in msg), msg
    return status == BAD


# ------------------------------------------------------------------ rotary
class View:
    """A strided view of elements of a buffer: offset and strides in elements."""

    def __init__(self, buf, at, b, h, n):
        self.buf, self.at, self.st = buf, at, (b, h, n)


def rotary(q, qo, k, ko, *, B=2, H=4, Hkv=2, N=10, d=64, elem=2, pos=None, freq=BASE + (9 << 32)):
    def ptr(v):
        return BASE + (v.buf << 32) + v.at * elem

    qs, ks = ((ctypes.c_longlong * 6)(*x.st, *y.st) for x, y in ((q, qo), (k, ko)))
    return refused("fa_rotary" if elem == 2 else "fa_rotary_f32",
                   [ptr(q), ptr(qo), ptr(k), ptr(ko), freq, pos, 0, B, H, Hkv, N, d, d, 0, 0, 1.0,
                    qs, ks, None])


def dense(buf, heads, N=10, d=64, at=0):
    return View(buf, at, heads * N * d, N * d, d)


def fused(buf, first, heads, N=10, d=64):
    """Heads from ``first`` on of a [B, N, heads, d] buffer."""
    return View(buf, first * d, N * heads * d, d, heads * d)


@no_gpu
@pytest.mark.parametrize("elem", [2, 4])
def test_rotary_layouts_that_share_nothing(elem):
    q, k = fused(0, 0, 8), fused(0, 4, 8)
    kw = {"elem": elem}
    assert not rotary(dense(0, 4), dense(1, 4), dense(2, 2), dense(3, 2), **kw)
    # heads of one fused buffer, both in place, one of them, or neither
    assert not rotary(q, q, k, k, **kw)
    assert not rotary(q, q, k, dense(1, 2), **kw)
    assert not rotary(q, dense(1, 4), k, k, **kw)
    assert not rotary(q, fused(1, 0, 8), k, fused(1, 4, 8), **kw)
    # queries turned into heads of the buffer that nothing else uses
    assert not rotary(fused(0, 0, 16), fused(0, 8, 16), fused(0, 4, 16), fused(0, 4, 16), **kw)
    # head-major: [B, heads, N, d] of both, one after the other in every sequence
    q, k = View(0, 0, 6 * 640, 640, 64), View(0, 4 * 640, 6 * 640, 640, 64)
    assert not rotary(q, q, k, k, **kw)
    # the same with a pitch between sequences that is no multiple of a token's
    q, k = View(0, 0, 10 * 512 + 72, 64, 512), View(0, 256, 10 * 512 + 72, 64, 512)
    assert not rotary(q, q, k, k, **kw)
    assert not rotary(q, q, k, dense(1, 2), **kw)
    # and one between heads of tokens side by side: [B, heads, N, 2, d]
    q, k = View(0, 0, 5 * 1288, 1288, 128), View(0, 64, 5 * 1288, 1288, 128)
    assert not rotary(q, q, k, k, H=4, Hkv=4, **kw)
    # one token in place: the token's own stride says nothing
    assert not rotary(dense(0, 4, N=1), View(0, 0, 256, 64, 9999), dense(1, 2, N=1), dense(2, 2, N=1),
                      N=1, **kw)
    # query and key of a head side by side: [B, N, heads, 2, d]
    q, k = View(0, 0, 10 * 512, 128, 512), View(0, 64, 10 * 512, 128, 512)
    assert not rotary(q, q, k, k, H=4, Hkv=4, **kw)


@no_gpu
@pytest.mark.parametrize("elem", [2, 4])
def test_rotary_outputs_over_other_arguments(elem):
    x, f = dense(0, 4), fused(0, 0, 8)
    kw = {"elem": elem}
    # the same tensor as query, in place, and as key, elsewhere: read while it is written
    assert rotary(x, x, x, dense(1, 4), H=4, Hkv=4, **kw)
    assert rotary(x, dense(1, 4), x, x, H=4, Hkv=4, **kw)
    assert rotary(f, f, f, dense(1, 4), H=4, Hkv=4, **kw)
    # heads that both tensors have, in place: turned twice
    assert rotary(f, f, fused(0, 3, 8), fused(0, 3, 8), **kw)
    assert rotary(x, x, View(0, 640, *x.st), View(0, 640, *x.st), **kw)
    p = View(0, 0, 10 * 512 + 72, 64, 512)
    assert rotary(p, p, View(0, 192, *p.st), View(0, 192, *p.st), **kw)
    assert rotary(p, p, View(0, 512, *p.st), View(0, 512, *p.st), **kw)
    # outputs with heads in common
    assert rotary(dense(0, 4), fused(2, 0, 8), dense(1, 2), fused(2, 3, 8), **kw)
    assert rotary(dense(0, 4), dense(2, 4), dense(1, 2), dense(2, 2, at=100), **kw)
    # one element in common
    assert rotary(dense(0, 4), dense(2, 4), dense(1, 2), dense(2, 2, at=2 * 4 * 640 - 1), **kw)


@no_gpu
def test_rotary_output_rows_that_share_elements():
    q, k = dense(0, 4), dense(2, 2)
    for st in ((2560, 64, 64), (2560, 640, 32), (64, 640, 64), (640, 640, 64), (0, 640, 64),
               (2559, 640, 64)):
        assert rotary(q, View(1, 0, *st), k, dense(3, 2))
    for st in ((2560, 640, 64), (64, 640, 2560 * 8), (64, 128, 512), (1 << 30, 640, 64)):
        assert not rotary(q, View(1, 0, *st), k, dense(3, 2))


def elements(v, heads, B, N, d):
    b, h, n, e = np.ogrid[:B, :heads, :N, :d]
    return (v.at + b * v.st[0] + h * v.st[1] + n * v.st[2] + e).ravel()


@no_gpu
def test_rotary_views_against_their_elements():
    """Random small views of one buffer: what shares an element is always refused, and what
    is laid out as one of the usual permutations of (batch, head, token) mostly is not."""
    rng = np.random.default_rng(1)
    accepted = apart = 0
    for _ in range(3000):
        B, H, Hkv, N, d = (int(rng.integers(1, m)) for m in (4, 5, 4, 6, 7))
        d += d % 2
        total, pad = H + Hkv + int(rng.integers(0, 3)), [int(x) for x in rng.integers(0, 3, 3)]
        order = rng.permutation(3)  # the dimensions from the innermost out
        st, step = [0, 0, 0], d + pad[0]
        for k, p in zip(order, (*pad[1:], 0)):
            st[k] = step
            step = step * (B, total, N)[k] + p
        if rng.random() < 0.2:
            st[int(rng.integers(0, 3))] = int(rng.integers(0, 2 * d))
        q = View(0, 16, *st)
        k = View(0, 16 + int(rng.choice([H * st[1], st[1], int(rng.integers(-12, 60))])), *st)
        out = [elements(q, H, B, N, d), elements(k, Hkv, B, N, d)]
        shares = (len(np.unique(out[0])) < out[0].size or len(np.unique(out[1])) < out[1].size or
                  np.intersect1d(*out).size > 0)
        got = rotary(q, q, k, k, B=B, H=H, Hkv=Hkv, N=N, d=d)
        assert got or not shares, (B, H, Hkv, N, d, st, k.at)
        apart += not shares
        accepted += not got
    assert accepted > 0.9 * apart > 500, (accepted, apart)


@no_gpu
def test_rotary_output_over_positions_and_frequencies():
    args = dense(0, 4), dense(1, 4), dense(2, 2), dense(3, 2)
    end = BASE + (1 << 32) + 2 * 4 * 640 * 2
    assert not rotary(*args, pos=end) and rotary(*args, pos=end - 4)
    assert not rotary(*args, freq=end) and rotary(*args, freq=end - 4)


# ------------------------------------------------------------------ paged cache
TREE = {"Q": 1, "K": 2, "V": 3, "O": 4, "LSE": 5, "table": 6, "lens": 7, "sq": 8, "mask": 9,
        "ws": 10}
# B=3 H=4 Hkv=2 T=5 pages=50 page=16 max_pages=20 d=64
TREE_BYTES = {"Q": 3 * 4 * 5 * 128, "K": 50 * 2 * 16 * 128, "V": 50 * 2 * 16 * 128,
              "O": 3 * 4 * 5 * 128, "LSE": 3 * 4 * 5 * 4, "table": 3 * 20 * 4, "lens": 12,
              "sq": 12, "mask": 3 * 5 * 8}


def tree(**at):
    ptr = {n: at.get(n, BASE + (i << 32)) for n, i in TREE.items()}
    need = binding.tree_workspace_bytes(3, 4, 2, 5, 64)
    return refused("fa_fwd_tree", [*list(ptr.values())[:9], 3, 4, 2, 5, 50, 16, 20, 64, 0.1, 0.0,
                                   ptr["ws"], need, None])


@no_gpu
@pytest.mark.parametrize("out", ["O", "LSE", "ws"])
def test_tree_outputs_over_other_arguments(out):
    assert not tree() and not tree(sq=None, mask=None, LSE=None)
    size = dict(TREE_BYTES, ws=binding.tree_workspace_bytes(3, 4, 2, 5, 64))
    for name, i in TREE.items():
        if name == out:
            continue
        at = BASE + (i << 32)
        last = at + (size[name] - 1) // 16 * 16  # (aligned as every output has to be)
        behind = at + (size[name] + 15) // 16 * 16
        assert tree(**{out: at}), name
        assert tree(**{out: last}), name
        assert not tree(**{out: behind}), name
        # and from in front
        mine = (size[out] + 15) // 16 * 16
        assert tree(**{out: at - mine + 16}) == (size[out] > mine - 16), name
        assert not tree(**{out: at - mine}), name


# ------------------------------------------------------------------ modified scores
MOD = {"Q": 1, "K": 2, "V": 3, "O": 4, "LSE": 5, "slopes": 6, "prefix": 7, "start": 8, "end": 9,
       "dO": 10, "dQ": 11, "dK": 12, "dV": 13, "ws": 14}
# B=3 H=4 Hkv=2 Nq=20 Nk=50 d=64
MOD_BYTES = {**dict.fromkeys(("Q", "O", "dO", "dQ"), 3 * 4 * 20 * 128),
             **dict.fromkeys(("K", "V", "dK", "dV"), 3 * 2 * 50 * 128), "LSE": 3 * 4 * 20 * 4,
             "slopes": 16, "prefix": 12, "start": 3 * 50 * 4, "end": 3 * 50 * 4}
SIZES = [3, 4, 2, 20, 50, 64, 0.1, 1, 0.0]


def mod(backward, **at):
    p = {n: at.get(n, BASE + (i << 32)) for n, i in MOD.items()}
    mods = [p[n] for n in ("slopes", "prefix", "start", "end")]
    if not backward:
        return refused("fa_fwd_mod", [*(p[n] for n in ("Q", "K", "V", "O", "LSE")), *mods, *SIZES,
                                      None])
    return refused("fa_bwd_mod", [*(p[n] for n in ("Q", "K", "V", "O", "dO", "LSE", "dQ", "dK", "dV")),
                                  *mods, *SIZES, p["ws"], binding.workspace_bytes(3, 4, 20, 64),
                                  None])


@no_gpu
@pytest.mark.parametrize("backward,out", [(False, "O"), (False, "LSE"), (True, "dQ"), (True, "dK"),
                                          (True, "dV"), (True, "ws")])
def test_mod_outputs_over_other_arguments(backward, out):
    assert not mod(backward)
    assert not mod(backward, slopes=None, prefix=None, start=None, end=None)
    size = dict(MOD_BYTES, ws=binding.workspace_bytes(3, 4, 20, 64))
    for name, i in MOD.items():
        if name == out or (not backward and name in ("dO", "dQ", "dK", "dV", "ws")):
            continue
        at = BASE + (i << 32)
        assert mod(backward, **{out: at}), name
        assert mod(backward, **{out: at + (size[name] - 1) // 16 * 16}), name
        assert not mod(backward, **{out: at + (size[name] + 15) // 16 * 16}), name
        assert not mod(backward, **{out: at - (size[out] + 15) // 16 * 16}), name


@no_gpu
def test_zeroed_key_gradients_over_keys():
    """Without queries dK and dV are zeroed: not over K or V."""
    def empty(**at):
        p = {n: at.get(n, BASE + (i << 32)) for n, i in MOD.items()}
        return refused("fa_bwd_mod", [*(p[n] for n in ("Q", "K", "V", "O", "dO", "LSE", "dQ", "dK", "dV")),
                                      None, None, None, None, 3, 4, 2, 0, 50, 64, 0.1, 1, 0.0, None, 0,
                                      None])

    assert not empty()
    for out, over in (("dK", "K"), ("dK", "V"), ("dV", "K"), ("dV", "V"), ("dK", "dV")):
        assert empty(**{out: BASE + (MOD[over] << 32)})
