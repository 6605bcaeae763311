"""The training operators' C entry points check their arguments on the host.

Runs without a GPU: every call here is refused before any CUDA call.
"""

import ctypes as C

import pytest

from speculative_decoding_head_gb300 import binding, build

EINVAL = 1
OK = C.c_void_p(256)     # never dereferenced: the checks come first
ODD = C.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _lce(**kw):
    a = {**dict(N=8, K=16, V=32, layout=0, ldx=16, ldw=16, ldu=32, lddx=16, lddw=16), **kw}
    return binding.LceDims(*(a[f] for f, _ in binding.LceDims._fields_))


def test_linear_ce_arguments(lib):
    def fwd(d, **kw):
        a = {**dict(X=OK, W=OK, U=OK, t=OK, loss=OK, lse=OK, scratch=OK, st=OK), **kw}
        return lib.dspark_linear_ce(C.byref(d) if d else None, a["X"], a["W"], a["U"], a["t"], a["loss"], a["lse"],
                                    a["scratch"], a["st"], None)

    def grad(d, **kw):
        a = {**dict(X=OK, W=OK, U=OK, t=OK, lse=OK, wt=OK, dX=OK, dW=OK, scratch=OK, st=OK), **kw}
        return lib.dspark_linear_ce_grad(C.byref(d) if d else None, a["X"], a["W"], a["U"], a["t"], a["lse"], a["wt"],
                                         1.0, a["dX"], a["dW"], a["scratch"], a["st"], None)

    bad_dims = [dict(N=-1), dict(K=0), dict(V=0), dict(layout=2), dict(N=(1 << 20) + 1), dict(K=65537),
                dict(V=(1 << 24) + 1), dict(ldx=15), dict(ldx=20), dict(ldw=8), dict(ldu=31), dict(ldu=34),
                dict(layout=1, ldw=24)]
    for kw in bad_dims:
        assert fwd(_lce(**kw)) == EINVAL, kw
        assert grad(_lce(**kw)) == EINVAL, kw
    assert fwd(None) == EINVAL and grad(None) == EINVAL
    for name in ("X", "W", "t", "loss", "lse", "scratch", "st"):
        assert fwd(_lce(), **{name: None}) == EINVAL, name
    for name in ("X", "W", "U", "t", "loss", "lse", "scratch"):
        assert fwd(_lce(), **{name: ODD}) == EINVAL, name
    for name in ("X", "W", "t", "lse", "scratch", "st"):
        assert grad(_lce(), **{name: None}) == EINVAL, name
    for name in ("X", "W", "U", "t", "lse", "wt", "dX", "dW", "scratch"):
        assert grad(_lce(), **{name: ODD}) == EINVAL, name
    assert grad(_lce(), dX=None, dW=None) == EINVAL
    assert grad(_lce(lddx=12)) == EINVAL and grad(_lce(lddw=12)) == EINVAL
    assert lib.dspark_linear_ce_scratch_bytes(None) == 0
    assert lib.dspark_linear_ce_scratch_bytes(C.byref(_lce(K=0))) == 0
    # the scratch grows with the rows, not with rows x vocabulary
    small = lib.dspark_linear_ce_scratch_bytes(C.byref(_lce(N=4096, K=256, V=129280)))
    assert 0 < small < 4096 * 129280 * 2


def test_embed_arguments(lib):
    def look(**kw):
        a = {**dict(E=OK, type=1, lde=16, V=20, D=16, idx=OK, N=8, out=OK, ldo=16, st=OK), **kw}
        return lib.dspark_embed(a["E"], a["type"], a["lde"], a["V"], a["D"], a["idx"], a["N"], 1.0, a["out"], a["ldo"],
                                a["st"], None)

    def grad(**kw):
        a = {**dict(dout=OK, type=1, ldd=16, idx=OK, N=8, V=20, D=16, base=None, ldb=16, dE=C.c_void_p(512), gtype=0,
                    lde=16, scratch=OK, st=OK), **kw}
        return lib.dspark_embed_grad(a["dout"], a["type"], a["ldd"], a["idx"], a["N"], a["V"], a["D"], 1.0, a["base"],
                                     a["ldb"], a["dE"], a["gtype"], a["lde"], a["scratch"], a["st"], None)

    odd = C.c_void_p(257)
    for kw in (dict(E=None), dict(out=None), dict(idx=None), dict(st=None), dict(type=2), dict(lde=15), dict(ldo=15),
               dict(V=0), dict(D=0), dict(N=-1), dict(N=(1 << 24) + 1), dict(E=odd), dict(idx=odd)):
        assert look(**kw) == EINVAL, kw
    for kw in (dict(dout=None), dict(dE=None), dict(idx=None), dict(st=None), dict(scratch=None), dict(type=2),
               dict(gtype=-1), dict(ldd=15), dict(lde=15), dict(base=OK, ldb=15), dict(V=0), dict(D=0), dict(N=-1),
               dict(dout=odd), dict(dE=odd), dict(base=odd), dict(scratch=ODD),
               dict(base=C.c_void_p(512), ldb=24)):
        assert grad(**kw) == EINVAL, kw
    assert look(N=0, E=None, out=None, idx=None) == 0        # no rows: nothing to do
    assert lib.dspark_embed_grad_scratch_bytes(-1, 20, 16) == 0
    assert lib.dspark_embed_grad_scratch_bytes(1000, 20, 16) > 0


def test_clip_arguments(lib):
    def clip(n=1, ptr=256, out=256, numel=10, type=0, max_norm=1.0, **kw):
        a = {**dict(norm=OK, scratch=OK, st=OK), **kw}
        arr = lambda t, v: (t * 1)(v)  # noqa: E731
        return lib.dspark_clip_grads(n, arr(C.c_void_p, ptr), arr(C.c_void_p, out), arr(C.c_int64, numel),
                                     arr(C.c_int32, type), max_norm, a["norm"], a["scratch"], a["st"], None)

    for kw in (dict(n=-1), dict(ptr=None), dict(out=None), dict(ptr=258), dict(ptr=257, type=1), dict(numel=-1),
               dict(type=2), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None), dict(scratch=None),
               dict(st=None), dict(scratch=C.c_void_p(260)), dict(numel=(1 << 44) + 1)):
        assert clip(**kw) == EINVAL, kw
    assert lib.dspark_clip_grads(1, None, None, None, None, 1.0, OK, OK, OK, None) == EINVAL
    assert lib.dspark_clip_grads_scratch_bytes(-1) == 0
    assert lib.dspark_clip_grads_scratch_bytes(513) == 2 * lib.dspark_clip_grads_scratch_bytes(512)
