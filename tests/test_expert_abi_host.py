"""CPU-only checks of the expert layer's and 8-bit products' entry points:
invalid arguments are refused on the host before anything touches a GPU, empty
calls are no-ops, and refusals come as SgemmError through check()."""
import pytest

FAKE = 1 << 40  # a never-dereferenced, 16-byte aligned address


@pytest.fixture(scope="module")
def lib():
    from dense_fp32_matrix_03_gb300 import build
    build.build()
    import dense_fp32_matrix_03_gb300 as m
    m.load()
    return m


def call(lib, name, **kw):
    spec = {
        "sgemm_i8_quantize_rows": dict(type_=0, act=0, M=4, K=8, X=FAKE, ldx=16, Q=FAKE, ldq=8,
                                       scale=FAKE),
        "sgemm_i8": dict(type_=0, M=4, N=4, K=8, A=FAKE, lda=8, scaleA=FAKE, B=FAKE, ldb=8,
                         scaleB=FAKE, C=FAKE, ldc=4),
        "sgemm_i8_experts": dict(type_=0, M=4, N=4, K=8, E=2, offsets=FAKE, A=FAKE, lda=8,
                                 scaleA=FAKE, B=FAKE, ldb=8, strideB=32, scaleB=FAKE, C=FAKE,
                                 ldc=4),
        "sgemm_experts_sort": dict(T=4, k=2, E=3, ids=FAKE, offsets=FAKE, slots=FAKE,
                                   positions=FAKE),
        "sgemm_experts_dispatch": dict(type_=0, T=4, k=2, E=3, H=8, x=FAKE, ldx=8, positions=FAKE,
                                       offsets=FAKE, rows=FAKE, ldr=8),
        "sgemm_experts_dispatch_i8": dict(type_=0, T=4, k=2, E=3, H=8, x=FAKE, ldx=8,
                                          positions=FAKE, offsets=FAKE, q=FAKE, ldq=8,
                                          scale=FAKE),
        "sgemm_experts_dispatch_grad": dict(type_=0, T=4, k=2, E=3, H=8, drows=FAKE, ldr=8,
                                            positions=FAKE, offsets=FAKE, dx=FAKE, ldx=8),
        "sgemm_experts_combine": dict(type_=0, T=4, k=2, E=3, H=8, rows=FAKE, ldr=8,
                                      positions=FAKE, offsets=FAKE, weights=FAKE, out=FAKE,
                                      ldo=8),
        "sgemm_experts_combine_grad": dict(type_=0, T=4, k=2, E=3, H=8, dout=FAKE, ldo=8,
                                           rows=FAKE, ldr=8, positions=FAKE, offsets=FAKE,
                                           weights=FAKE, drows=FAKE, ldd=8, dweights=FAKE),
    }[name]
    assert set(kw) <= set(spec), kw
    return getattr(lib, name)(**{**spec, **kw})


ROWS = ["sgemm_experts_dispatch", "sgemm_experts_dispatch_i8", "sgemm_experts_dispatch_grad",
        "sgemm_experts_combine", "sgemm_experts_combine_grad"]
BAD = [
    *[("sgemm_i8_quantize_rows", b) for b in (
        dict(type_=3), dict(type_=-1), dict(act=2), dict(M=-1), dict(K=-1), dict(ldx=7),
        dict(act=1, K=9, ldx=17, ldq=9), dict(ldq=7), dict(X=0), dict(X=FAKE + 1),
        dict(type_=2, X=FAKE + 2), dict(Q=0), dict(scale=0), dict(scale=FAKE + 2))],
    *[("sgemm_i8", b) for b in (
        dict(type_=3), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=7), dict(ldb=7), dict(ldc=3),
        dict(A=0), dict(B=0), dict(C=0), dict(C=FAKE + 1), dict(scaleA=0), dict(scaleB=0),
        dict(scaleA=FAKE + 1), dict(scaleB=FAKE + 2), dict(K=131072, lda=131072, ldb=131072))],
    *[("sgemm_i8_experts", b) for b in (
        dict(E=0), dict(E=1025), dict(offsets=0), dict(offsets=FAKE + 2), dict(strideB=-1),
        dict(strideB=31), dict(type_=7), dict(lda=7))],
    *[("sgemm_experts_sort", b) for b in (
        dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(ids=0), dict(offsets=0),
        dict(slots=0), dict(positions=0), dict(ids=FAKE + 1), dict(T=2 ** 30, k=2),
        dict(positions=FAKE + 2))],
    *[(n, b) for n in ROWS for b in (
        dict(type_=3), dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(H=-1),
        dict(H=9), dict(positions=0), dict(offsets=0), dict(positions=FAKE + 1),
        dict(offsets=FAKE + 2), dict(T=2 ** 30))],
    *[("sgemm_experts_dispatch", b) for b in (dict(x=0), dict(rows=0), dict(x=FAKE + 1))],
    *[("sgemm_experts_dispatch_i8", b) for b in (dict(x=0), dict(q=0), dict(scale=0))],
    *[("sgemm_experts_dispatch_grad", b) for b in (dict(drows=0), dict(dx=0), dict(ldx=7))],
    *[("sgemm_experts_combine", b) for b in (dict(rows=0), dict(out=0), dict(weights=FAKE + 2),
                                             dict(type_=2, out=FAKE + 2))],
    *[("sgemm_experts_combine_grad", b) for b in (
        dict(dout=0), dict(drows=0), dict(rows=0), dict(ldr=7), dict(dweights=FAKE + 1))],
]


@pytest.mark.parametrize("name,bad", BAD)
def test_invalid_arguments_are_refused(lib, name, bad):
    assert call(lib, name, **bad) == lib.SGEMM_ERR_INVALID_ARG
    with pytest.raises(lib.SgemmError):
        lib.check(call(lib, name, **bad))


@pytest.mark.parametrize("name,empty", [
    ("sgemm_i8_quantize_rows", dict(M=0, X=0, Q=0, scale=0)),
    ("sgemm_i8", dict(M=0)), ("sgemm_i8", dict(N=0)), ("sgemm_i8_experts", dict(M=0)),
    *[(n, dict(T=0)) for n in ROWS],
    ("sgemm_experts_combine", dict(H=0, rows=0, out=0)),
])
def test_empty_calls_do_nothing(lib, name, empty):
    assert call(lib, name, **empty) == lib.SGEMM_OK


def test_names_of_types_and_acts(lib):
    assert call(lib, "sgemm_i8_quantize_rows", type_="bf16", act="none", M=0) == lib.SGEMM_OK
    with pytest.raises(KeyError):
        call(lib, "sgemm_i8", type_="int8")


@pytest.mark.parametrize("name", ["sgemm_i8", "sgemm_i8_experts"])
def test_sides_end_where_a_tile_past_them_is_still_an_int(lib, name):
    most = 2 ** 31 - 512
    more = dict(strideB=8 * (most + 1)) if name == "sgemm_i8_experts" else {}
    for side in ("M", "N"):
        kw = dict(ldc=most + 1, **more)
        assert call(lib, name, **{side: most + 1}, **kw) == lib.SGEMM_ERR_INVALID_ARG
