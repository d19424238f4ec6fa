"""Host-side checks of the C ABI of linear attention and of trees of drafted tokens (no GPU needed): every
invalid call returns its documented status before anything is enqueued, and the bindings refuse tensors
that the C calls could not check."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from gated_deltanet_hybrid_amd import hla

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL_ARG, BAD_SHAPE, BAD_DTYPE, WORKSPACE, HIP, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 5, 6, 7
P, PU, P4 = 0x10000, 0x10008, 0x10004  # placeholder addresses, never dereferenced
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return hla.library()


def dims(**kw):
    f = dict(B=2, T=200, H=4, Hk=2, ld_T=256, dk=128, dv=64, dtype=1, decay_per_head=0)
    f.update(kw)
    return ctypes.byref(hla._LaDims(*f.values()))


BAD_DIMS = [(dict(dtype=2), BAD_DTYPE), (dict(dtype=-1), BAD_DTYPE), (dict(B=0), BAD_SHAPE), (dict(T=0), BAD_SHAPE),
            (dict(H=0, Hk=0), BAD_SHAPE), (dict(Hk=0), BAD_SHAPE), (dict(Hk=3), BAD_SHAPE), (dict(Hk=8), BAD_SHAPE),
            (dict(ld_T=199), BAD_SHAPE), (dict(dk=96), BAD_SHAPE), (dict(dv=256), BAD_SHAPE),
            (dict(decay_per_head=2), BAD_SHAPE), (dict(H=65537, Hk=65537), BAD_SHAPE), (dict(B=1 << 22), BAD_SHAPE),
            (dict(T=1 << 37, ld_T=1 << 37), BAD_SHAPE), (dict(B=1 << 20, ld_T=1 << 34), BAD_SHAPE)]


# (d, q, k, v, log_decay, lens, S0, o, S_final, ws, ws_bytes, stream)
FWD = [None, P, P, P, P, P, P, P, P, P, BIG, None]
# (d, q, k, v, log_decay, lens, S0, dO, dS_final, dq, dk, dv, dlog_decay, dS0, ws, ws_bytes, stream)
BWD = [None, P, P, P, P, P, P, P, P, P, P, P, P, P, P, BIG, None]


@pytest.mark.parametrize("kw,status", BAD_DIMS, ids=str)
def test_dims(lib, kw, status):
    d, n = dims(**kw), ctypes.c_size_t()
    for fn in (0, 1):
        assert lib.hla_la_workspace_bytes(fn, d, ctypes.byref(n)) == status
    assert lib.hla_la_prefill(d, *FWD[1:]) == status
    assert lib.hla_la_prefill_backward(d, *BWD[1:]) == status


def test_prefill_arguments(lib):
    def put(i, x):
        a = list(FWD)
        a[0], a[i] = dims(), x
        return lib.hla_la_prefill(*a)

    assert lib.hla_la_prefill(None, *FWD[1:]) == NULL_ARG
    for i in (2, 3, 4):
        assert put(i, None) == NULL_ARG
    a = list(FWD)
    a[0], a[1] = dims(), None
    assert lib.hla_la_prefill(*a) == NULL_ARG          # o without q
    a[1], a[7], a[8] = P, None, None
    assert lib.hla_la_prefill(*a) == NULL_ARG          # no output
    for i in (1, 2, 3, 6, 7, 8, 9):
        assert put(i, PU) == ALIGN
    for i in (4, 5):
        assert put(i, P + 2) == ALIGN
    assert put(10, 16) == WORKSPACE                    # two rows of four pieces are cut in two
    assert put(9, None) == WORKSPACE


def test_backward_arguments(lib):
    def put(i, x):
        a = list(BWD)
        a[0], a[i] = dims(), x
        return lib.hla_la_prefill_backward(*a)

    assert lib.hla_la_prefill_backward(None, *BWD[1:]) == NULL_ARG
    for i in (1, 2, 3, 4, 7, 9, 10, 11, 12):
        assert put(i, None) == NULL_ARG
    for i in (1, 2, 3, 6, 7, 8, 9, 10, 11, 13, 14):
        assert put(i, PU) == ALIGN
    for i in (4, 5, 12):
        assert put(i, P + 2) == ALIGN
    n = ctypes.c_size_t()
    assert lib.hla_la_workspace_bytes(1, dims(), ctypes.byref(n)) == OK and n.value > 0
    assert put(15, n.value - 1) == WORKSPACE and put(14, None) == WORKSPACE


def test_workspace_bytes(lib):
    n = ctypes.c_size_t()
    assert lib.hla_la_workspace_bytes(0, dims(), None) == NULL_ARG
    assert lib.hla_la_workspace_bytes(2, dims(), ctypes.byref(n)) == UNSUPPORTED
    # many rows, or one piece: one segment, nothing kept
    for kw in (dict(B=512, H=8, Hk=8), dict(T=64)):
        assert lib.hla_la_workspace_bytes(0, dims(**kw), ctypes.byref(n)) == OK and n.value == 0
    # one row of 64 pieces of 64 tokens: a float32 state and a float64 sum for each of its segments
    assert lib.hla_la_workspace_bytes(0, dims(B=1, H=1, Hk=1, T=4096, ld_T=4096), ctypes.byref(n)) == OK
    segments = n.value // (128 * 64 * 4)
    assert 2 <= segments <= 64 and n.value == segments * 128 * 64 * 4 + -(-segments * 8 // 256) * 256
    # the sum over shared heads counts its threads in 32 bits
    assert lib.hla_la_workspace_bytes(1, dims(B=64, T=1 << 20, ld_T=1 << 20), ctypes.byref(n)) == BAD_SHAPE
    assert lib.hla_la_workspace_bytes(1, dims(B=64, T=1 << 20, ld_T=1 << 20, Hk=4), ctypes.byref(n)) == OK


def test_decode_arguments(lib):
    # (Bs, H, Hk, dk, dv, dtype, q, k, v, log_decay, per_head, S, o, stream)
    a = [2, 4, 2, 128, 64, 1, P4, P4, P4, P4, 0, P, P4, None]
    put = lambda i, x: lib.hla_la_decode(*(a[:i] + [x] + a[i + 1:]))  # noqa: E731
    for i, x in ((0, 0), (1, 0), (2, 3), (3, 32), (4, 0), (10, 2), (0, 1 << 23)):
        assert put(i, x) == BAD_SHAPE
    assert put(5, 7) == BAD_DTYPE
    for i in (6, 7, 8, 9, 11, 12):
        assert put(i, None) == NULL_ARG
    assert put(11, PU) == ALIGN
    for i in (6, 7, 8, 9, 12):
        assert put(i, P + 2) == ALIGN


# (Bs, H, n, dk, dv, dtype, q, k, v, beta, alpha, parent, S_cur, At_cur, At_cache, Bc_cache, reps, n_rep, n_cache, n_cap,
#  gates_in, tau, o, gates_out, ws, ws_bytes, stream)
TREE = [2, 3, 7, 128, 64, 1, P, P, P, P4, P4, P4, P, P, P, P, P, 2, P4, 5, None, 0.1, P, P4, P, BIG, None]
# (Bs, H, n, dk, dv, dtype, k, v, beta, alpha, parent, node, S_cur, At_cur, At_cache, Bc_cache, n_cache, n_cap, commit, stream)
ACCEPT = [2, 3, 7, 128, 64, 1, P, P, P4, P4, P4, P4, P, P, P, P, P4, 5, P4, None]
SIZES = ((0, 0), (1, 0), (2, 0), (2, 65), (3, 96), (4, 32), (0, 1 << 23))


def test_tree_decode_arguments(lib):
    put = lambda i, x: lib.hla_gdn_tree_decode(*(TREE[:i] + [x] + TREE[i + 1:]))  # noqa: E731
    for i, x in SIZES + ((19, 0), (19, 1025), (17, 0), (17, -1), (21, float("nan"))):
        assert put(i, x) == BAD_SHAPE, (i, x)
    assert put(5, 3) == BAD_DTYPE
    for i in (6, 7, 8, 9, 10, 11, 12, 14, 15, 16, 18, 22):
        assert put(i, None) == NULL_ARG, i
    for i in (6, 7, 8, 12, 13, 14, 15, 16, 22, 24):
        assert put(i, PU) == ALIGN, i
    for i in (9, 10, 11, 18, 20, 23):
        assert put(i, P + 2) == ALIGN, i
    need = hla.gdn_tree_workspace_bytes(2, 3, 7, 128, 64, 5)
    assert need >= 6 * (7 * 128 + 5 * 7 + 5) * 4
    assert put(25, need - 1) == WORKSPACE and put(24, None) == WORKSPACE


def test_tree_workspace_bytes(lib):
    n = ctypes.c_size_t()
    f = lib.hla_gdn_tree_workspace_bytes
    assert f(2, 3, 7, 128, 64, 5, None) == NULL_ARG
    for a in ((0, 3, 7, 128, 64, 5), (2, 3, 65, 128, 64, 5), (2, 3, 7, 128, 64, -1), (2, 3, 7, 128, 64, 1025)):
        assert f(*a, ctypes.byref(n)) == BAD_SHAPE
    assert f(2, 3, 7, 128, 64, 0, ctypes.byref(n)) == OK and n.value == 0


def test_tree_accept_arguments(lib):
    put = lambda i, x: lib.hla_gdn_tree_accept(*(ACCEPT[:i] + [x] + ACCEPT[i + 1:]))  # noqa: E731
    for i, x in SIZES + ((17, 0), (17, 1025)):
        assert put(i, x) == BAD_SHAPE, (i, x)
    assert put(5, -1) == BAD_DTYPE
    for i in (6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16):  # 13 ..: what commit needs
        assert put(i, None) == NULL_ARG, i
    for i in (6, 7, 12, 13, 14, 15):
        assert put(i, PU) == ALIGN, i
    for i in (8, 9, 10, 11, 16, 18):
        assert put(i, P + 2) == ALIGN, i


def la_tensors(**kw):
    t = dict(q=torch.zeros(2, 9, 2, 64), k=torch.zeros(2, 9, 2, 64), v=torch.zeros(2, 9, 4, 128), g=torch.zeros(2, 9, 4))
    t.update(kw)
    return t["q"], t["k"], t["v"], t["g"]


@pytest.mark.parametrize("kw", [dict(v=torch.zeros(2, 9, 128)), dict(k=torch.zeros(2, 8, 2, 64)),
                                dict(k=torch.zeros(2, 9, 2, 64, dtype=torch.bfloat16)), dict(q=torch.zeros(2, 9, 4, 64)),
                                dict(g=torch.zeros(2, 9, 2)), dict(g=torch.zeros(3)), dict(g=torch.zeros(2, 9, 4).double()),
                                dict(q=torch.zeros(2, 2, 9, 64).transpose(1, 2)), dict(k=torch.zeros(2, 12, 2, 64)[:, 3:])],
                         ids=range(9))
def test_bindings_refuse_layouts(kw):
    a = la_tensors(**kw)
    with pytest.raises(ValueError):
        hla.la_prefill(*a)
    with pytest.raises(ValueError):
        hla.la_prefill_backward(*a, torch.zeros(2, 9, 4, 128))


def test_bindings_refuse_other_arguments():
    a = la_tensors()
    for kw in (dict(lens=torch.zeros(2)), dict(lens=torch.zeros(3, dtype=torch.int32)), dict(S0=torch.zeros(2, 4, 128, 64)),
               dict(o=torch.zeros(2, 9, 4, 128).bfloat16()), dict(S_final=torch.zeros(2, 4, 64, 128).double()),
               dict(ws=torch.zeros(4))):
        with pytest.raises(ValueError):
            hla.la_prefill(*a, **kw)
    for dO in (torch.zeros(2, 9, 4, 64), torch.zeros(2, 9, 4, 128).bfloat16(), torch.zeros(2, 18, 4, 128)[:, ::2]):
        with pytest.raises(ValueError):
            hla.la_prefill_backward(*a, dO)
    with pytest.raises(ValueError):
        hla.la_decode(torch.zeros(2, 2, 64), torch.zeros(2, 2, 64), torch.zeros(2, 4, 128), torch.zeros(2, 4), torch.zeros(2, 4, 128, 64))
    with pytest.raises(TypeError):
        hla.la_prefill(*(x.half() if x.dim() == 4 else x for x in a))


def tree_tensors():
    return dict(k=torch.zeros(2, 5, 3, 64), v=torch.zeros(2, 5, 3, 128), beta=torch.zeros(2, 5, 3), alpha=torch.zeros(2, 5, 3),
                parent=torch.zeros(2, 5, dtype=torch.int32), S_cur=torch.zeros(2, 3, 64, 128))


@pytest.mark.parametrize("name,bad", [("k", torch.zeros(2, 5, 64)), ("v", torch.zeros(2, 4, 3, 128)),
                                      ("beta", torch.zeros(2, 3, 5)), ("alpha", torch.zeros(2, 5, 3).double()),
                                      ("parent", torch.zeros(2, 5)), ("S_cur", torch.zeros(2, 3, 128, 64))])
def test_bindings_refuse_trees(name, bad):
    t = tree_tensors()
    t[name] = bad
    with pytest.raises(ValueError):
        hla.gdn_tree_decode(torch.zeros(2, 5, 3, 64), **t)
    node = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        hla.gdn_tree_accept(t["k"], t["v"], t["beta"], t["alpha"], t["parent"], node, t["S_cur"])


def test_bindings_refuse_accept_without_its_cache():
    t = tree_tensors()
    node = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        hla.gdn_tree_accept(t["k"], t["v"], t["beta"], t["alpha"], t["parent"], node, t["S_cur"], commit=node)
    with pytest.raises(ValueError):
        hla.gdn_tree_accept(t["k"], t["v"], t["beta"], t["alpha"], t["parent"], node.long(), t["S_cur"])


def test_host_code_sanitized(tmp_path):
    """These checks again, with the host code built with ASan and UBSan."""
    from test_abi_sanitized import _asan_runtime

    from gated_deltanet_hybrid_amd import build
    rt = _asan_runtime()
    if rt is None or "HLA_LIBRARY" in os.environ:
        pytest.skip("no shared ASan runtime, or the sanitized run itself")
    if not all(os.path.exists(os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o")) for s in build.SOURCES):
        pytest.skip("the library's objects are not built")
    lib = build.build_host_sanitized(str(tmp_path / "libhla_san.so"))
    env = dict(os.environ, HLA_LIBRARY=lib, LD_PRELOAD=rt, PYTHONPATH=ROOT + os.pathsep + os.path.join(ROOT, "tests"),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-p", "no:cacheprovider"], env=env,
                       capture_output=True, text=True, timeout=600, cwd=str(tmp_path))
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
