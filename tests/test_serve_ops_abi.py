"""The C entry points of the 4-bit matrices and of sampling check their arguments on the host.

Runs without a GPU: every call here is refused before any CUDA call, or has nothing to do.
"""

import ctypes as C

import pytest

from speculative_decoding_head_gb300 import binding, build

EINVAL = 1
OK = 256                 # never dereferenced: the checks come first
ODD = 264


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _dims(**kw):
    a = {**dict(rows=8, K=64, format=0), **kw}
    return C.byref(binding.Fp4Dims(a["rows"], a["K"], a["format"]))


def _data(**kw):
    a = {**dict(codes=OK, scales=OK, rowf=OK), **kw}
    return C.byref(binding.Fp4Data(a["codes"], a["scales"], a["rowf"]))


BAD_DIMS = [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(K=0), dict(K=65537), dict(format=2), dict(format=-1)]
BAD_DATA = [dict(codes=None), dict(scales=None), dict(rowf=None), dict(codes=ODD), dict(scales=ODD), dict(rowf=260)]


def test_fp4_sizes(lib):
    for kw in BAD_DIMS:
        assert lib.dspark_fp4_code_bytes(_dims(**kw)) == 0 and lib.dspark_fp4_scale_bytes(_dims(**kw)) == 0
    assert lib.dspark_fp4_code_bytes(None) == 0 and lib.dspark_fp4_scale_bytes(None) == 0
    assert lib.dspark_fp4_code_bytes(_dims(rows=3, K=33)) == 3 * 32
    # whole groups of 128 rows and of 256 columns: a byte for 16 columns, or for 32
    assert lib.dspark_fp4_scale_bytes(_dims(rows=129, K=257)) == 256 * 32
    assert lib.dspark_fp4_scale_bytes(_dims(rows=129, K=257, format=1)) == 256 * 16
    # counted in 64 bits
    assert lib.dspark_fp4_code_bytes(_dims(rows=1 << 24, K=65536)) == 1 << 39


def test_fp4_quant_arguments(lib):
    def f(d=None, m=None, **kw):
        a = {**dict(X=OK, type=1, ldx=64, count=None, st=OK), **kw}
        return lib.dspark_fp4_quant(d or _dims(), a["X"], a["type"], a["ldx"], a["count"], m or _data(), a["st"], None)

    for kw in BAD_DIMS:
        assert f(d=_dims(**kw)) == EINVAL, kw
    for kw in BAD_DATA:
        assert f(m=_data(**kw)) == EINVAL, kw
    for kw in (dict(X=None), dict(X=257), dict(X=258, type=0), dict(type=2), dict(ldx=63), dict(st=None),
               dict(count=258)):
        assert f(**kw) == EINVAL, kw
    assert lib.dspark_fp4_quant(None, OK, 1, 64, None, _data(), OK, None) == EINVAL
    assert lib.dspark_fp4_quant(_dims(), OK, 1, 64, None, None, OK, None) == EINVAL
    assert f(d=_dims(rows=0), X=None) == 0


def test_fp4_rows_arguments(lib):
    def f(d=None, m=None, **kw):
        a = {**dict(idx=OK, N=5, out=OK, type=1, ldo=64, st=OK), **kw}
        return lib.dspark_fp4_rows(d or _dims(), m or _data(), a["idx"], a["N"], a["out"], a["type"], a["ldo"], a["st"],
                                   None)

    for kw in BAD_DIMS + [dict(rows=0)]:
        assert f(d=_dims(**kw)) == EINVAL, kw
    for kw in BAD_DATA:
        assert f(m=_data(**kw)) == EINVAL, kw
    for kw in (dict(N=-1), dict(N=(1 << 24) + 1), dict(idx=None, N=9), dict(idx=258), dict(out=None), dict(out=257),
               dict(out=258, type=0), dict(type=-1), dict(ldo=63), dict(st=None)):
        assert f(**kw) == EINVAL, kw
    assert f(N=0, out=None) == 0


def test_fp4_linear_arguments(lib):
    def f(xd=None, x=None, wd=None, w=None, **kw):
        a = {**dict(U=OK, ldu=16, Y=512, type=0, ldy=16, st=OK), **kw}
        return lib.dspark_fp4_linear(xd or _dims(), x or _data(), wd or _dims(rows=16), w or _data(), a["U"], a["ldu"],
                                     a["Y"], a["type"], a["ldy"], a["st"], None)

    for kw in BAD_DIMS:
        assert f(xd=_dims(**kw)) == EINVAL and f(wd=_dims(**kw)) == EINVAL, kw
    for kw in BAD_DATA:
        assert f(x=_data(**kw)) == EINVAL and f(w=_data(**kw)) == EINVAL, kw
    assert f(wd=_dims(rows=0)) == EINVAL
    assert f(wd=_dims(rows=16, K=32)) == EINVAL              # another K
    assert f(wd=_dims(rows=16, format=1)) == EINVAL          # another format
    for kw in (dict(U=258), dict(ldu=15), dict(Y=None), dict(Y=514), dict(Y=513, type=1), dict(type=2), dict(ldy=15),
               dict(st=None), dict(U=512, ldu=17), dict(U=512, type=1)):
        assert f(**kw) == EINVAL, kw
    assert f(xd=_dims(rows=0), Y=None) == 0


def _args(**kw):
    a = {**dict(N=8, V=64, requests=0, type=0, ldz=64, row_off=None, temperature=None, top_k=None, top_p=None,
                min_p=None), **kw}
    return C.byref(binding.SampleArgs(*(a[f] for f, _ in binding.SampleArgs._fields_)))


def test_sample_arguments(lib):
    def draw(d=None, **kw):
        a = {**dict(Z=OK, u=OK, token=OK, logp=OK, st=OK), **kw}
        return lib.dspark_sample(d or _args(), a["Z"], a["u"], a["token"], a["logp"], a["st"], None)

    def dist(d=None, **kw):
        a = {**dict(Z=OK, fill=0.0, out=512, ldo=64, st=OK), **kw}
        return lib.dspark_sample_logprobs(d or _args(), a["Z"], a["fill"], a["out"], a["ldo"], a["st"], None)

    for kw in (dict(N=-1), dict(N=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(type=2), dict(ldz=63),
               dict(row_off=OK), dict(row_off=258, requests=2), dict(temperature=258), dict(top_k=257), dict(top_p=259),
               dict(min_p=258)):
        assert draw(_args(**kw)) == EINVAL and dist(_args(**kw)) == EINVAL, kw
    for kw in (dict(Z=None), dict(Z=258), dict(st=None)):
        assert draw(**kw) == EINVAL and dist(**kw) == EINVAL, kw
    for kw in (dict(u=None), dict(u=258), dict(token=None), dict(token=257), dict(logp=258)):
        assert draw(**kw) == EINVAL, kw
    for kw in (dict(out=None), dict(out=514), dict(ldo=63), dict(out=OK)):
        assert dist(**kw) == EINVAL, kw
    assert draw(_args(type=1), Z=257) == EINVAL
    assert lib.dspark_sample(None, OK, OK, OK, OK, OK, None) == EINVAL
    assert lib.dspark_sample_logprobs(None, OK, 0.0, OK, 64, OK, None) == EINVAL
    assert draw(_args(N=0), Z=None, u=None, token=None) == 0 and dist(_args(N=0), Z=None, out=None) == 0
