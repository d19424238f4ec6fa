"""Host-side checks of the 8-bit chunk cache's C ABI and of its oracle (no GPU needed): every
invalid call returns its documented status before anything is enqueued."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import oracle.cache8 as o8
from gated_deltanet_hybrid_amd import hla

OK, NULL_ARG, BAD_SHAPE, BAD_DTYPE, WORKSPACE, HIP, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 5, 6, 7
P, PU = 0x10000, 0x10008  # placeholder addresses, aligned to 16 bytes and to 8; never dereferenced


@pytest.fixture(scope="module")
def lib():
    return hla.library()


def cache(**kw):
    f = dict(Bs=1, H=2, dk=128, dv=64, n_cap=4, n_rep=2, format=0, maps=P, reps=P, scale=P, order=P, count=P, weight=P)
    f.update(kw)
    return ctypes.byref(hla._Cache8Struct(*f.values()))


BAD_CACHES = [(dict(format=2), BAD_DTYPE), (dict(format=-1), BAD_DTYPE), (dict(Bs=0), BAD_SHAPE), (dict(H=0), BAD_SHAPE),
              (dict(dk=96), BAD_SHAPE), (dict(dv=0), BAD_SHAPE), (dict(n_cap=0), BAD_SHAPE), (dict(n_cap=1025), BAD_SHAPE),
              (dict(n_rep=-1), BAD_SHAPE), (dict(n_rep=257), BAD_SHAPE), (dict(Bs=1 << 31), BAD_SHAPE),
              (dict(maps=None), NULL_ARG), (dict(reps=None), NULL_ARG), (dict(scale=None), NULL_ARG),
              (dict(order=None), NULL_ARG), (dict(count=None), NULL_ARG), (dict(maps=PU), ALIGN), (dict(reps=PU), ALIGN),
              (dict(scale=PU), ALIGN), (dict(order=P + 2), ALIGN), (dict(weight=P + 1), ALIGN)]


def calls(lib, c):
    n = ctypes.c_size_t()
    yield lib.hla_decode8_workspace_bytes(c, ctypes.byref(n))
    yield lib.hla_gdn_decode8(c, 1, P, P, P, P, P, P, P, None, 0.0, P, None, P, 1 << 40, None)
    yield lib.hla_gdn2_decode8(c, 1, P, P, P, P, P, P, P, P, None, 0.0, P, None, P, 1 << 40, None)
    yield lib.hla_cache8_append(c, 1, 1, 1, P, P, P, 2, None, None, None, 0, 0, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=str)
def test_every_call_checks_the_cache(lib, kw, status):
    assert list(calls(lib, cache(**kw))) == [status] * 4


def test_null_cache(lib):
    assert list(calls(lib, None)) == [NULL_ARG] * 4
    assert lib.hla_decode8_workspace_bytes(cache(), None) == NULL_ARG


def test_decode8_validation(lib):
    f1, f2 = lib.hla_gdn_decode8, lib.hla_gdn2_decode8
    # (cache, dtype, q, k, v, beta, alpha, S_cur, At_cur, gates_in, tau, o, gates_out, ws, ws_bytes, stream)
    a1 = [cache(), 1, P, P, P, P, P, P, P, None, 0.0, P, None, P, 1 << 40, None]
    a2 = a1[:6] + [P] + a1[6:]
    for f, a, tau in ((f1, a1, 10), (f2, a2, 11)):
        put = lambda i, x: f(*(a[:i] + [x] + a[i + 1:]))  # noqa: E731
        assert put(1, 2) == BAD_DTYPE
        assert put(tau, float("nan")) == BAD_SHAPE
        for i in [*range(2, tau - 1), tau + 1]:
            assert put(i, None) == NULL_ARG, i
            assert put(i, P + 2) == ALIGN, i
        assert put(tau - 3, PU) == put(tau - 2, PU) == ALIGN  # the live matrices move in 16-byte vectors
        assert put(tau - 1, P + 2) == put(tau + 2, P + 1) == ALIGN
        assert put(tau + 3, PU) == ALIGN
        none = cache(n_rep=0, reps=None)
        assert f(none, *a[1:]) == NULL_ARG  # no representatives and no gates


def test_decode8_workspace(lib):
    n = ctypes.c_size_t()
    for Bs, H, n_cap in itertools.product((1, 3, 256), (1, 16), (1, 64, 1024)):
        assert lib.hla_decode8_workspace_bytes(cache(Bs=Bs, H=H, n_cap=n_cap), ctypes.byref(n)) == OK
        if n.value:
            a = [cache(Bs=Bs, H=H, n_cap=n_cap), 1, P, P, P, P, P, P, P, None, 0.0, P, None]
            assert lib.hla_gdn_decode8(*a, None, n.value, None) == WORKSPACE
            assert lib.hla_gdn_decode8(*a, P, n.value - 1, None) == WORKSPACE


def test_append_validation(lib):
    f = lib.hla_cache8_append
    # (cache, dtype, n_src, ld_src, At, Bc, reps, ld_R, src, n_new, weight_in, reset, reset_live, stream)
    a = [cache(), 0, 3, 5, P, P, P, 6, None, None, None, 0, 0, None]
    put = lambda *kv: f(*[dict(kv).get(i, x) for i, x in enumerate(a)])  # noqa: E731
    assert put((1, 2)) == BAD_DTYPE
    assert put((2, -1)) == put((2, 6)) == put((2, 0), (3, 0)) == put((3, 2)) == BAD_SHAPE
    assert put((11, 2)) == put((12, -1)) == BAD_SHAPE
    assert put((7, 5)) == put((7, 1 << 62)) == BAD_SHAPE  # rows that are not there, or not addressable
    assert f(cache(Bs=1 << 30, H=1), 0, 3, 1 << 30, *a[4:]) == BAD_SHAPE
    for i in (4, 5, 6):
        assert put((i, None)) == NULL_ARG
        assert put((i, PU)) == ALIGN
    for i in (8, 9, 10):
        assert put((i, P + 2)) == ALIGN
    assert put((8, P), (12, 1)) == UNSUPPORTED
    assert put((1, 1), (12, 1)) == UNSUPPORTED


def test_gate_weights_and_evict_validation(lib):
    g = lib.hla_gate_weights
    assert g(0, 1, 1, P, None, 0.0, P, None) == g(1, 0, 1, P, None, 0.0, P, None) == g(1, 1, 0, P, None, 0.0, P, None) == BAD_SHAPE
    assert g(1 << 31, 1, 1, P, None, 0.0, P, None) == g(1, 1, 1, P, None, float("nan"), P, None) == BAD_SHAPE
    assert g(1, 1, 1, None, None, 0.0, P, None) == g(1, 1, 1, P, None, 0.0, None, None) == NULL_ARG
    assert g(1, 1, 1, P + 2, None, 0.0, P, None) == g(1, 1, 1, P, P + 1, 0.0, P, None) == ALIGN
    e = lib.hla_evict_chunks
    # (Bs, H, n, weight, order, count, budget, n_recent, order_out, weight_out, count_out, stream)
    a = [1, 1, 4, P, None, P, 2, 1, P, P, P, None]
    put = lambda *kv: e(*[dict(kv).get(i, x) for i, x in enumerate(a)])  # noqa: E731
    assert put((0, 0)) == put((1, 0)) == put((2, 0)) == put((2, 16385)) == put((0, 1 << 31)) == BAD_SHAPE
    assert put((6, -1)) == put((7, -1)) == put((7, 3)) == BAD_SHAPE
    for i in (3, 5, 8, 9, 10):
        assert put((i, None)) == NULL_ARG
        assert put((i, P + 2)) == ALIGN
    assert put((4, P + 2)) == ALIGN


def test_launches_are_counted_in_32_bits(lib):
    """Refused where a grid's threads would pass 32 bits, whatever memory would hold."""
    n = ctypes.c_size_t()
    for dk, dv in itertools.product((64, 128), repeat=2):
        rows = (1 << 32) // ((dk + dv) * 4)
        ok, over = cache(Bs=rows - 1, H=1, dk=dk, dv=dv), cache(Bs=rows + 1, H=1, dk=dk, dv=dv)
        assert lib.hla_decode8_workspace_bytes(ok, ctypes.byref(n)) == OK
        assert lib.hla_decode8_workspace_bytes(over, ctypes.byref(n)) == BAD_SHAPE
    assert lib.hla_cache8_append(cache(Bs=1 << 12, H=1 << 7), 1, 16, 16, P, P, P, 32, None, None, None, 0, 0, None) == BAD_SHAPE
    assert lib.hla_gate_weights(1 << 24, 1, 1, P, None, 0.0, P, None) == BAD_SHAPE
    for rows, n_pos in ((1 << 26, 1), (1 << 26, 256), (1 << 24, 257), (1 << 24, 4096), (1 << 22, 4097)):
        assert lib.hla_evict_chunks(rows, 1, n_pos, P, None, P, 1, 1, P, P, P, None) == BAD_SHAPE


def test_python_refuses_host_tensors():
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        hla.Cache8(z(1, 1, 2, 128, 64, dt=torch.int8), None, z(1, 1, 2, 4), z(1, 1, 2, dt=torch.int32), z(1, 1, dt=torch.int32))


def test_oracle_stored_values():
    """The oracle's formats against their definitions: every e4m3 code, exact ties to the even
    code, the largest magnitude on the top value."""
    v = o8.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448 and np.all(np.diff(v) > 0)
    assert np.array_equal(v, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy())
    ties = (v[:-1] + v[1:]) / 2
    x = np.concatenate([ties, -ties, [448.0]]).astype(np.float32)
    q, s = o8.quantise(x, "e4m3")
    assert s == 1.0
    code = np.searchsorted(v, np.abs(q[:len(ties)]))
    assert np.all(code % 2 == 0) and np.array_equal(q[:len(ties)], -q[len(ties):-1])
    q, s = o8.quantise(np.array([127.0, 0.5, 1.5, -2.5, -126.5]), "int8")
    assert s == 1.0 and q.tolist() == [127, 0, 2, -2, -126]
    assert o8.quantise(np.full(3, 2.0 ** -101), "int8") == (pytest.approx([0, 0, 0]), 0.0)


def test_oracle_evict():
    o, w, c = o8.evict(np.array([3, 1, 1, 0, 9], np.float32), np.array([4, 2, 0, 1, 3]), 4, 2, 1)
    assert o.tolist() == [4, 1, 2, 0, 3] and w.tolist() == [3, 0, 0, 0, 0] and c == 2  # the newest stays, of 1, 1 both go
    o, w, c = o8.evict(np.array([1, np.nan, 1, 2], np.float32), np.arange(4), 4, 2, 0)
    assert o.tolist() == [2, 3, 0, 1] and w.tolist() == [1, 2, 0, 0] and c == 2


def test_python_refuses_host_arrays():
    with pytest.raises(ValueError):
        hla.gate_weights(torch.zeros(1, 1, 2, 2))
    with pytest.raises(ValueError):
        hla.evict_chunks(torch.zeros(1, 1, 2), torch.zeros(1, 1, dtype=torch.int32), 1)
    with pytest.raises(KeyError):
        hla.cache8_alloc(1, 1, 2, 64, 64, fmt="int4")
