"""The serving entry points on the host: argument checks before anything touches
the GPU, workspace sizes, and the rotary frequencies and tables."""
import ctypes
import math

import numpy as np
import pytest
import torch

from helpers import spa

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, NOMEM = 0, 1, 2, 3, 4, 5, 6
F32, BF16 = 0, 1
A = 0x100000  # an aligned dummy address, never dereferenced by validation


@pytest.fixture(scope="module")
def lib():
    return spa().lib


def rope(lib, q=A, k=A, qo=A, ko=A, strides=None, pos=A, pos0=0, table=A, B=2, H=4, Hk=2, N=8, d=64,
         rot=64, inter=0, inv=0, scale=1.0, dtype=BF16):
    if strides is not None:
        strides = (ctypes.c_longlong * 12)(*strides)
    return lib.spa_rope(q, k, qo, ko, strides, pos, pos0, table, B, H, Hk, N, d, rot, inter, inv,
                        scale, dtype, None)


def test_rope_rejects_bad_arguments(lib):
    assert rope(lib, q=None) == NULL
    assert rope(lib, ko=None) == NULL
    assert rope(lib, table=None) == NULL
    assert rope(lib, B=-1) == SHAPE
    assert rope(lib, dtype=2) == DTYPE
    assert rope(lib, d=0, rot=2) == UNSUPPORTED
    assert rope(lib, d=1025, rot=2) == UNSUPPORTED
    for rot in (0, 7, 66, -2):
        assert rope(lib, rot=rot) == SHAPE
    assert rope(lib, q=A + 1) == ALIGN
    assert rope(lib, q=A + 2, dtype=F32) == ALIGN
    assert rope(lib, table=A + 4) == ALIGN
    assert rope(lib, pos=A + 2) == ALIGN
    assert rope(lib, pos=None, pos0=2**31 - 7) == SHAPE        # the last row's position overflows
    assert rope(lib, B=2**15, N=2**15) == SHAPE
    assert rope(lib, q=None, k=None, qo=None, ko=None, table=None, N=0) == OK
    assert rope(lib, q=None, k=None, qo=None, ko=None, table=None, H=0, Hk=0) == OK


def test_rope_rejects_overlapping_output_rows(lib):
    dense_q, dense_k = (4 * 8 * 64, 8 * 64, 64), (2 * 8 * 64, 8 * 64, 64)
    B = A + (1 << 24)
    def call(qo=dense_q, ko=dense_k, q=dense_q, out=B):
        return rope(lib, strides=(*q, *dense_k, *qo, *ko), qo=out, ko=B + (1 << 20))
    assert call(qo=(0, 8 * 64, 64)) == SHAPE              # two sequences on the same rows
    assert call(qo=(4 * 8 * 64, 8 * 64, 63)) == SHAPE     # rows that run into one another
    assert call(qo=(4 * 8 * 64, 7 * 64, 64)) == SHAPE     # heads that do
    assert call(ko=(2 * 8 * 64, -8 * 64, 64)) == SHAPE
    assert call(q=(0, 8 * 64, 64), out=A) == SHAPE        # in place, but with other strides


def append(lib, k=A, v=A, P=A, kc=A, mul=A, vc=A, pos=A, count=None, acc=None, row_pos=None,
           token=None, B=2, H=2, T=3, d=64, m=32, dv=64, cap=16, dtype=BF16):
    return lib.spa_kcache_append_ragged(k, v, P, kc, mul, vc, pos, count, acc, row_pos, token, B, H,
                                        T, d, m, dv, cap, dtype, None)


def test_append_rejects_bad_arguments(lib):
    for name in ("k", "v", "P", "kc", "mul", "vc", "pos"):
        assert append(lib, **{name: None}) == NULL
    for name in ("k", "v", "P", "kc", "vc"):
        assert append(lib, **{name: A + 8}) == ALIGN
    for name in ("mul", "pos", "count", "acc", "row_pos", "token"):
        assert append(lib, **{name: A + 2}) == ALIGN
    assert append(lib, T=-1) == SHAPE
    assert append(lib, B=300, H=300) == SHAPE
    assert append(lib, dtype=F32) == UNSUPPORTED
    assert append(lib, dtype=3) == DTYPE
    assert append(lib, d=257) == UNSUPPORTED
    assert append(lib, m=48) == UNSUPPORTED
    assert append(lib, dv=32) == UNSUPPORTED
    assert append(lib, k=None, v=None, P=None, kc=None, mul=None, vc=None, pos=None, T=0) == OK


def decode(lib, q=A, P=A, kc=A, mul=A, v=A, lens=A, pkc=A, pmul=A, pv=A, out=A, acc=None, acc_out=None,
           B=2, H=4, Hk=2, plen=8, pcap=8, d=64, m=32, dv=64, cap=16, dtype=BF16, ws=A, size=1 << 30):
    return lib.spa_attention_decode_shared(q, P, kc, mul, v, lens, pkc, pmul, pv, out, acc, acc_out, B,
                                           H, Hk, plen, pcap, d, m, dv, cap, dtype, ws, size, None)


def test_decode_rejects_bad_arguments(lib):
    for name in ("q", "P", "kc", "mul", "v", "lens", "pkc", "pmul", "pv", "out"):
        assert decode(lib, **{name: None}) == NULL
    for name in ("q", "P", "kc", "v", "pkc", "pv", "out"):
        assert decode(lib, **{name: A + 8}) == ALIGN
    for name in ("mul", "lens", "pmul"):
        assert decode(lib, **{name: A + 2}) == ALIGN
    assert decode(lib, acc=A) == NULL and decode(lib, acc_out=A) == NULL   # both or neither
    assert decode(lib, ws=A + 128) == ALIGN
    assert decode(lib, size=0) == NOMEM
    assert decode(lib, pcap=7) == SHAPE            # more prefix rows than it holds
    assert decode(lib, plen=-1) == SHAPE
    assert decode(lib, H=3) == SHAPE               # heads that do not share evenly
    assert decode(lib, Hk=0) == SHAPE
    assert decode(lib, B=30000) == SHAPE
    assert decode(lib, dtype=F32) == UNSUPPORTED
    assert decode(lib, dtype=7) == DTYPE
    assert decode(lib, d=300) == UNSUPPORTED
    assert decode(lib, m=8) == UNSUPPORTED
    assert decode(lib, dv=96) == UNSUPPORTED
    assert decode(lib, q=None, P=None, out=None, B=0) == OK


def test_decode_workspace_size(lib):
    n = ctypes.c_size_t(7)
    size = lib.spa_attention_decode_shared_workspace_size
    assert size(2, 4, 2, 8, 64, 32, 64, 16, 0, ctypes.byref(n)) == OK and n.value > 0
    plain = n.value
    assert size(2, 4, 2, 8, 64, 32, 64, 16, 1, ctypes.byref(n)) == OK and n.value > plain
    assert size(0, 4, 2, 8, 64, 32, 64, 16, 1, ctypes.byref(n)) == OK and n.value == 0
    assert size(2, 3, 2, 8, 64, 32, 64, 16, 1, ctypes.byref(n)) == SHAPE
    assert size(2, 4, 2, 8, 64, 32, 64, 16, 1, None) == NULL


def evict(lib, kc=A, mul=A, v=A, acc=A, row_pos=A, lens=A, acc_out=A, pos_out=A, lens_out=A, src=A, B=2,
          H=2, m=32, dv=64, cap=64, budget=16, sink=1, recent=4, ws=A, size=1 << 30):
    return lib.spa_kcache_evict(kc, mul, v, acc, row_pos, lens, acc_out, pos_out, lens_out, src, B, H, m,
                                dv, cap, budget, sink, recent, ws, size, None)


def test_evict_rejects_bad_arguments(lib):
    for name in ("kc", "mul", "v", "acc", "row_pos", "lens", "acc_out", "pos_out", "lens_out", "src"):
        assert evict(lib, **{name: None}) == NULL
    for name in ("kc", "v"):
        assert evict(lib, **{name: A + 8}) == ALIGN
    for name in ("mul", "acc", "row_pos", "lens", "acc_out", "pos_out", "lens_out", "src"):
        assert evict(lib, **{name: A + 2}) == ALIGN
    assert evict(lib, budget=0) == SHAPE
    assert evict(lib, budget=65) == SHAPE
    assert evict(lib, sink=-1) == SHAPE
    assert evict(lib, recent=-1) == SHAPE
    assert evict(lib, sink=13, recent=4) == SHAPE
    assert evict(lib, B=300, H=300) == SHAPE
    assert evict(lib, m=33) == UNSUPPORTED
    assert evict(lib, cap=2**20 + 1) == UNSUPPORTED
    assert evict(lib, dv=65) == UNSUPPORTED
    assert evict(lib, size=16) == NOMEM
    assert evict(lib, ws=A + 16) == ALIGN
    assert evict(lib, kc=None, src=None, B=0) == OK


def test_rope_frequencies():
    pkg = spa()
    rot, base = 16, 10000.0
    want = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    f = pkg.rope_frequencies(rot, base).numpy()
    assert np.allclose(f, want, rtol=1e-14, atol=0)
    f = pkg.rope_frequencies(rot, base, pkg.SPA_ROPE_LINEAR, factor=4.0).numpy()
    assert np.allclose(f, want / 4, rtol=1e-14, atol=0)
    f = pkg.rope_frequencies(rot, base, pkg.SPA_ROPE_BASE, factor=4.0).numpy()
    assert math.isclose(f[0], 1.0) and math.isclose(f[-1], want[-1] / 4, rel_tol=1e-12)
    trained, slow, fast = 512.0, 1.0, 8.0
    f = pkg.rope_frequencies(rot, base, pkg.SPA_ROPE_RAMP, factor=4.0, trained=trained, slow=slow,
                             fast=fast).numpy()
    turns = trained * want / (2 * math.pi)
    keep = np.clip((turns - slow) / (fast - slow), 0, 1)
    assert np.allclose(f, keep * want + (1 - keep) * want / 4, rtol=1e-13, atol=0)
    assert (keep == 1).any() and (keep == 0).any() and ((keep > 0) & (keep < 1)).any()
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, base=math.inf),
                dict(rot=8, scaling=1, factor=0.0), dict(rot=2, scaling=2, factor=2.0),
                dict(rot=8, scaling=3, factor=2.0), dict(rot=8, scaling=9),
                dict(rot=8, scaling=3, factor=2.0, trained=9.0, slow=4.0, fast=4.0)):
        with pytest.raises(pkg.SpaError):
            pkg.rope_frequencies(**bad)


def test_rope_table_is_the_fraction_of_a_turn():
    pkg = spa()
    f = torch.tensor([1.0, 0.5 ** 40, math.pi, 2 * math.pi * 3, 100.0, -1.0], dtype=torch.float64)
    t = pkg.rope_table(f, device="cpu").tolist()
    for fi, ti in zip(f.tolist(), t):
        turns = fi / (2 * math.pi)
        part = turns - round(turns)
        # the same fraction up to the rounding of the double
        off = (ti / 2.0**64 - part) % 1.0
        assert min(off, 1 - off) < 2.0**-52 * max(1.0, abs(turns))
    with pytest.raises(pkg.SpaError):
        pkg.rope_table([math.nan], device="cpu")
    with pytest.raises(ValueError):
        pkg.rope_table(torch.ones(2, 2), device="cpu")


def test_binding_refuses_host_tensors():
    pkg = spa()
    q = torch.zeros((1, 2, 3, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.spa_rope(q, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        pkg.spa_kcache_append_ragged(q, q, q, q, q, q, q)
    with pytest.raises(ValueError):
        pkg.spa_attention_decode_shared(q[:, :, 0], q, q, q, q, q)
    with pytest.raises(ValueError):
        pkg.spa_kcache_evict(q, q, q, q, q, q, 1)


def test_decode_selftest_arguments():
    pkg = spa()
    assert pkg.selftest_decode_wait_timeout(0, 0) == SHAPE
    assert pkg.selftest_decode_wait_timeout(2001, 1) == SHAPE
    assert pkg.selftest_decode_wait_timeout(50, 2) == UNSUPPORTED
    assert pkg.selftest_decode_wait_timeout(50, -1) == UNSUPPORTED
