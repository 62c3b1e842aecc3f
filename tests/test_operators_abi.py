"""Host-side checks of the modified-score, rotary and paged-cache calls (no GPU: every call
here is refused, or finishes, before a device is touched), and the float64 gradient that
the modified-score kernels are held to against differences."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import mod_reference as ref
from exact_io_aware_64_b200 import binding

BAD, UNSUP, OK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_OK
P = [0x1000000 * (i + 1) for i in range(16)]  # 16-byte aligned, 16 MB apart


def call(fn, names, defaults, **kw):
    a = dict(zip(names, defaults))
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    lib = binding.lib()
    st = getattr(lib, fn)(*a.values())
    return st, lib.fa_last_error_message().decode()


FWD = ("Q K V O LSE slopes prefix start end B H Hkv Nq Nk d scale causal cap stream".split(),
       [P[0], P[1], P[2], P[3], P[4], None, None, None, None, 1, 4, 2, 16, 16, 64, 0.1, 0, 0.0,
        None])
BWD = ("Q K V O dO LSE dQ dK dV slopes prefix start end B H Hkv Nq Nk d scale causal cap ws "
       "ws_bytes stream".split(),
       [*P[:9], None, None, None, None, 1, 4, 2, 16, 16, 64, 0.1, 0, 0.0, P[9], 1 << 20, None])

MOD_BAD = [
    ({"Hkv": 3}, BAD), ({"Hkv": 0}, BAD), ({"Hkv": -1}, BAD), ({"H": 4, "Hkv": 8}, BAD),
    ({"cap": -1.0}, BAD), ({"cap": float("nan")}, BAD), ({"cap": float("inf")}, BAD),
    ({"cap": 1e-38}, BAD), ({"cap": 1e35}, BAD), ({"prefix": P[10], "causal": 0}, BAD),
    ({"start": P[10]}, BAD), ({"end": P[10]}, BAD), ({"start": P[10] + 2, "end": P[11]}, BAD),
    ({"slopes": P[10] + 1}, BAD), ({"prefix": P[10] + 2, "causal": 1}, BAD), ({"d": 96}, UNSUP),
    ({"causal": 1, "Nq": 17}, BAD), ({"Nk": 0}, BAD), ({"scale": 0.0}, BAD), ({"Q": None}, BAD),
    ({"K": P[1] + 8}, BAD), ({"B": 1 << 15, "H": 1 << 12, "Hkv": 1, "Nq": 1 << 10}, BAD),
    ({"LSE": P[4] + 2}, BAD),
]


@pytest.mark.parametrize("kw,status", MOD_BAD)
def test_mod_refusals(kw, status):
    assert call("fa_fwd_mod", *FWD, **kw)[0] == status
    assert call("fa_bwd_mod", *BWD, **kw)[0] == status


def test_mod_overlaps_and_workspace():
    assert call("fa_fwd_mod", *FWD, O=P[0] + 16)[0] == BAD
    assert call("fa_fwd_mod", *FWD, O=P[2] + 16)[0] == BAD
    for kw in ({"dQ": P[0]}, {"dK": P[6]}, {"dV": P[1] + 16}, {"ws": P[7]}, {"ws": P[5]},
               {"ws": None}, {"ws_bytes": 8}, {"dV": None}):
        st, msg = call("fa_bwd_mod", *BWD, **kw)
        assert st == BAD and msg


def test_mod_empty_calls():
    for kw in ({"B": 0}, {"H": 0, "Hkv": 0}, {"Nq": 0, "Nk": 0}):
        null = dict.fromkeys("Q K V O LSE".split())
        assert call("fa_fwd_mod", *FWD, **null, **kw)[0] == OK
        assert call("fa_bwd_mod", *BWD, **null, **kw)[0] == OK
    assert call("fa_fwd_mod", *FWD, Nq=0)[0] == OK
    # keys without queries: the gradients are written, so they are checked
    assert call("fa_bwd_mod", *BWD, Nq=0, dK=None)[0] == BAD


def test_doc_ranges_refusals():
    names = "ids start end B N stream".split()
    d = [P[0], P[1], P[2], 2, 100, None]
    for kw in ({"ids": None}, {"start": None}, {"end": P[2] + 2}, {"B": -1}, {"N": -1},
               {"N": (1 << 30) + 1}, {"B": 1 << 16, "N": 1 << 16}, {"start": P[0] + 16},
               {"end": P[1]}):
        assert call("fa_doc_ranges", names, d, **kw)[0] == BAD
    assert call("fa_doc_ranges", names, d, B=0, ids=None)[0] == OK
    assert call("fa_doc_ranges", names, d, N=0)[0] == OK


ROT = ("Q Qo K Ko freq pos first B H Hkv N d R interleaved inverse mscale qs ks stream".split(),
       [P[0], P[1], P[2], P[3], P[4], None, 0, 2, 4, 2, 10, 64, 64, 0, 0, 1.0, None, None, None])


def strides(*s):
    return (ctypes.c_longlong * 6)(*s)


@pytest.mark.parametrize("fn", ["fa_rotary", "fa_rotary_f32"])
def test_rotary_refusals(fn):
    bad = [{"R": 63}, {"R": 66}, {"R": -2}, {"interleaved": 2}, {"inverse": -1},
           {"mscale": float("nan")}, {"B": -1}, {"N": -1}, {"H": -1}, {"Q": None}, {"Ko": None},
           {"freq": None}, {"freq": P[4] + 1}, {"pos": P[5] + 2}, {"Q": P[0] + 1},
           {"Qo": P[0] + 64}, {"Qo": P[3]}, {"B": 1 << 16, "N": 1 << 15}, {"first": 1 << 50},
           {"qs": strides(-1, 640, 64, 2560, 640, 64)}, {"qs": strides(2560, 640, 64, 2560, 640, 0)},
           {"qs": strides(1 << 41, 640, 64, 2560, 640, 64)},
           {"H": 1 << 28, "N": 1 << 6}, {"Qo": P[2] + 64}, {"Ko": P[0] + 64}, {"Qo": P[2]}]
    for kw in bad:
        st, msg = call(fn, *ROT, **kw)
        assert st == BAD and msg, kw
    assert call(fn, *ROT, d=514)[0] == UNSUP
    assert call(fn, *ROT, B=0)[0] == OK and call(fn, *ROT, N=0)[0] == OK
    assert call(fn, *ROT, H=0, Hkv=0, Q=None)[0] == OK
    # in place with nothing to turn
    assert call(fn, *ROT, R=0, Qo=P[0], Ko=P[2], freq=None)[0] == OK


TREE = ("Q K V O LSE table lens sq mask B H Hkv T num_pages page max_pages d scale cap ws "
        "ws_bytes stream".split(),
        [P[0], P[1], P[2], P[3], P[4], P[5], P[6], None, None, 2, 4, 2, 3, 50, 16, 20, 64, 0.1,
         0.0, P[7], 1 << 24, None])


def test_tree_refusals():
    bad = [{"Hkv": 3}, {"Hkv": 0}, {"B": -1}, {"T": -1}, {"scale": 0.0}, {"cap": -1.0},
           {"cap": float("nan")}, {"num_pages": -1}, {"max_pages": -1}, {"num_pages": 0},
           {"Q": None}, {"K": P[1] + 8}, {"O": P[0] + 16}, {"O": P[2]}, {"table": None},
           {"lens": None}, {"lens": P[6] + 2}, {"sq": P[8] + 1}, {"mask": P[8] + 4},
           {"LSE": P[4] + 2}, {"ws": None}, {"ws": P[7] + 8}, {"ws_bytes": 100}, {"ws": P[1]},
           {"page": 128, "max_pages": 1 << 24}, {"B": 4096, "max_pages": 1 << 20}]
    for kw in bad:
        st, msg = call("fa_fwd_tree", *TREE, **kw)
        assert st == BAD and msg, kw
    for kw in ({"d": 96}, {"T": 65}, {"page": 4}, {"page": 24}, {"page": 192}, {"page": 0},
               {"B": 4097}):
        st, msg = call("fa_fwd_tree", *TREE, **kw)
        assert st == UNSUP and msg, kw
    for kw in ({"B": 0}, {"H": 0, "Hkv": 0}, {"T": 0}):
        assert call("fa_fwd_tree", *TREE, **kw, Q=None, ws=None)[0] == OK


def test_tree_workspace():
    f = binding.tree_workspace_bytes
    assert f(0, 4, 2, 1, 64) == 0 and f(1, 4, 3, 1, 64) == 0
    assert f(1, 16, 4, 1, 128) >= (148 + 4) * 2 * 4 * 128 * 4
    assert f(2, 16, 2, 64, 128) >= (148 + 2 * 2 * 2) * 256 * 128 * 4
    assert f(1, 1, 1, 1, 64) < 1 << 20


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    f = torch.zeros(32)
    with pytest.raises(ValueError):
        binding.fwd_mod(x, x, x)
    with pytest.raises(ValueError):
        binding.doc_ranges(torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.rotary(x, None, f)
    with pytest.raises(ValueError):
        binding.rotary(x.half(), None, f)
    with pytest.raises(ValueError):
        binding.fwd_tree(x, x, x, torch.zeros(1, 1, dtype=torch.int32),
                         torch.zeros(1, dtype=torch.int32))
    for bad in ({"rot": 3}, {"rot": 0}, {"rot": 64, "factor": 0.0}, {"rot": 64, "scaling": "?"}):
        with pytest.raises(ValueError):
            binding.rotary_frequencies(device="cpu", **bad)


def test_gradient_against_differences():
    """The float64 gradient formula against central differences of the float64 forward, with
    every modification at once."""
    rng = np.random.default_rng(0)
    Q, K, V, G = (rng.standard_normal((9, 4)) for _ in range(4))
    ids = np.array([0, 0, 0, 0, 1, 1, 1, -1, -1])
    seen = ref.visible(9, 9, True, 3, ids)
    f = lambda: (ref.forward(Q, K, V, 0.5, seen, 1.5, 0.2)[0] * G).sum()  # noqa: E731
    for t, grad in zip((Q, K, V), ref.backward(Q, K, V, G, 0.5, seen, 1.5, 0.2)):
        for at in itertools.product(range(9), range(4)):
            old, h = t[at], 1e-6
            t[at] = old + h
            up = f()
            t[at] = old - h
            down = f()
            t[at] = old
            assert abs((up - down) / (2 * h) - grad[at]) < 1e-7
