"""CPU-only checks of the norm's, the 4-bit products' and the few-token expert
layer's entry points: invalid arguments are refused on the host before anything
touches a GPU, empty calls are no-ops, sizes are what the layouts need."""
import pytest

FAKE = 1 << 40  # a never-dereferenced, 16-byte aligned address


@pytest.fixture(scope="module")
def lib():
    from dense_fp32_matrix_03_gb300 import build
    build.build()
    import dense_fp32_matrix_03_gb300 as m
    m.load()
    return m


STREAM = dict(type_=0, M=4, H=8, eps=1e-5, x=FAKE, ldx=8, res=FAKE, ldr=8, weight=FAKE, sum_=FAKE,
              lds=8)
SPECS = {
    "sgemm_rms_norm": dict(STREAM, y=FAKE, ldy=8),
    "sgemm_rms_norm_i8": dict(STREAM, q=FAKE, ldq=8, scale=FAKE),
    "sgemm_rms_norm_fp4": dict(STREAM, format_=1, q=FAKE, ldq=32, sf=FAKE, scale=FAKE),
    "sgemm_rms_norm_grad": dict(type_=0, M=4, H=8, eps=1e-5, s=FAKE, lds=8, weight=FAKE, dy=FAKE,
                                ldy=8, dsum=FAKE, ldds=8, dx=FAKE, ldx=8, dweight=FAKE,
                                workspace=FAKE, workspace_bytes=4 * 8 * 4),
    "sgemm_fp4_quantize_rows": dict(type_=0, act=0, format_=0, M=4, K=8, X=FAKE, ldx=16, Q=FAKE,
                                    ldq=32, sf=FAKE, scale=FAKE),
    "sgemm_fp4": dict(type_=0, format_=1, M=4, N=4, K=40, A=FAKE, lda=64, sfA=FAKE, scaleA=FAKE,
                      B=FAKE, ldb=64, sfB=FAKE, scaleB=FAKE, C=FAKE, ldc=4),
    "sgemm_experts_layer": dict(type_=0, wtype=0, T=4, k=2, E=3, H=16, F=32, x=FAKE, ldx=16,
                                ids=FAKE, weights=FAKE, W1=FAKE, ld1=16, stride1=64 * 16,
                                scale1=FAKE, W2=FAKE, ld2=32, stride2=16 * 32, scale2=FAKE,
                                out=FAKE, ldo=16, workspace=FAKE, workspace_bytes=8 * 32 * 4),
}
NORMS = ["sgemm_rms_norm", "sgemm_rms_norm_i8", "sgemm_rms_norm_fp4"]


def call(lib, name, **kw):
    assert set(kw) <= set(SPECS[name]), kw
    return getattr(lib, name)(**{**SPECS[name], **kw})


BAD = [
    *[(n, b) for n in NORMS for b in (
        dict(type_=3), dict(type_=-1), dict(M=-1), dict(H=-1), dict(eps=0.0), dict(eps=-1.0),
        dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-40), dict(ldx=7), dict(ldr=7),
        dict(lds=7), dict(x=0), dict(x=FAKE + 1), dict(type_=2, x=FAKE + 2), dict(res=FAKE + 1),
        dict(weight=FAKE + 1), dict(sum_=FAKE + 1))],
    *[("sgemm_rms_norm", b) for b in (dict(y=0), dict(y=FAKE + 1), dict(ldy=7))],
    *[("sgemm_rms_norm_i8", b) for b in (dict(q=0), dict(ldq=7), dict(scale=0),
                                         dict(scale=FAKE + 2))],
    *[("sgemm_rms_norm_fp4", b) for b in (
        dict(format_=2), dict(format_=-1), dict(q=0), dict(q=FAKE + 8), dict(ldq=40), dict(ldq=0),
        dict(sf=0), dict(sf=FAKE + 4), dict(scale=0), dict(H=33, ldx=33, ldr=33, lds=33))],
    *[("sgemm_rms_norm_grad", b) for b in (
        dict(type_=3), dict(M=-1), dict(H=-1), dict(eps=0.0), dict(lds=7), dict(ldy=7),
        dict(ldds=7), dict(ldx=7), dict(s=0), dict(dy=0), dict(dx=0), dict(s=FAKE + 1),
        dict(dy=FAKE + 1), dict(dsum=FAKE + 1), dict(dx=FAKE + 1), dict(weight=FAKE + 1),
        dict(dweight=FAKE + 2), dict(workspace=0), dict(workspace=FAKE + 8),
        dict(workspace_bytes=127))],
    *[("sgemm_fp4_quantize_rows", b) for b in (
        dict(type_=3), dict(act=2), dict(format_=2), dict(M=-1), dict(K=-1), dict(ldx=7),
        dict(act=1, K=9, ldx=17), dict(ldq=31), dict(ldq=48), dict(K=33, ldx=33), dict(X=0),
        dict(X=FAKE + 1), dict(Q=0), dict(Q=FAKE + 8), dict(sf=0), dict(sf=FAKE + 8),
        dict(scale=0), dict(scale=FAKE + 2))],
    *[("sgemm_fp4", b) for b in (
        dict(type_=3), dict(format_=2), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=32),
        dict(lda=40), dict(ldb=32), dict(ldb=72), dict(ldc=3), dict(A=0), dict(B=0), dict(C=0),
        dict(sfA=0), dict(sfB=0), dict(A=FAKE + 8), dict(B=FAKE + 8), dict(sfA=FAKE + 4),
        dict(sfB=FAKE + 4), dict(C=FAKE + 1), dict(scaleA=FAKE + 2), dict(scaleB=FAKE + 2),
        dict(M=2 ** 31 - 511), dict(N=2 ** 31 - 511, ldc=2 ** 31 - 1),
        dict(K=2 ** 31 - 8191, lda=2 ** 31 - 32, ldb=2 ** 31 - 32))],
    *[("sgemm_experts_layer", b) for b in (
        dict(type_=2), dict(type_=3), dict(wtype=2), dict(T=-1), dict(T=65), dict(k=0),
        dict(T=64, k=9), dict(k=65), dict(E=0), dict(E=1025), dict(H=-1), dict(F=-1),
        dict(ldx=15), dict(ldo=15), dict(ld1=8), dict(ld1=24, wtype=0), dict(ld2=16),
        dict(ld2=40), dict(stride1=64 * 16 - 16), dict(stride2=16 * 32 - 16),
        dict(stride1=64 * 16 + 8), dict(stride2=-16), dict(x=0), dict(ids=0), dict(out=0),
        dict(W1=0), dict(W2=0), dict(scale1=0), dict(scale2=0), dict(workspace=0),
        dict(workspace_bytes=1023), dict(x=FAKE + 1), dict(out=FAKE + 1), dict(ids=FAKE + 2),
        dict(weights=FAKE + 2), dict(W1=FAKE + 8), dict(W2=FAKE + 8), dict(scale1=FAKE + 2),
        dict(workspace=FAKE + 8), dict(H=65537, ldx=65537, ldo=65537))],
]


@pytest.mark.parametrize("name,bad", BAD)
def test_invalid_arguments_are_refused(lib, name, bad):
    assert call(lib, name, **bad) == lib.SGEMM_ERR_INVALID_ARG
    with pytest.raises(lib.SgemmError):
        lib.check(call(lib, name, **bad))


@pytest.mark.parametrize("name,empty", [
    *[(n, dict(M=0, x=0)) for n in NORMS], ("sgemm_rms_norm", dict(H=0, x=0, y=0)),
    ("sgemm_rms_norm_grad", dict(M=0, dweight=0)), ("sgemm_rms_norm_grad", dict(H=0)),
    ("sgemm_fp4_quantize_rows", dict(M=0, X=0, Q=0, sf=0, scale=0)),
    ("sgemm_fp4", dict(M=0)), ("sgemm_fp4", dict(N=0)),
    ("sgemm_experts_layer", dict(T=0)), ("sgemm_experts_layer", dict(H=0)),
])
def test_empty_calls_do_nothing(lib, name, empty):
    assert call(lib, name, **empty) == lib.SGEMM_OK


def test_sizes(lib):
    assert lib.sgemm_fp4_scales_size("nv", 1, 1) == 512
    assert lib.sgemm_fp4_scales_size("nv", 129, 65) == 2 * 2 * 512
    assert lib.sgemm_fp4_scales_size("mx", 128, 128) == 512
    assert lib.sgemm_fp4_scales_size("mx", 128, 129) == 1024
    assert lib.sgemm_fp4_scales_size("mx", 2 ** 31 - 1, 2 ** 31 - 1) == 2 ** 24 * 2 ** 24 * 512
    assert lib.sgemm_fp4_scales_size("nv", 0, 64) == 0
    assert lib.sgemm_fp4_scales_size("mx", -1, 64) == 0
    assert lib.sgemm_fp4_scales_size(7, 4, 64) == 0
    assert lib.sgemm_rms_norm_grad_workspace_size(4, 8) == 4 * 8 * 4
    assert lib.sgemm_rms_norm_grad_workspace_size(10 ** 6, 8) == 608 * 8 * 4
    assert lib.sgemm_rms_norm_grad_workspace_size(-1, 8) == 0
    assert lib.sgemm_experts_layer_workspace_size(4, 2, 16, 33) == 8 * 48 * 4
    assert lib.sgemm_experts_layer_workspace_size(65, 1, 16, 16) == 0


def test_names_of_formats_and_weights(lib):
    assert call(lib, "sgemm_fp4", type_="fp16", format_="nv", M=0) == lib.SGEMM_OK
    assert call(lib, "sgemm_experts_layer", type_="bf16", wtype="same", T=0) == lib.SGEMM_OK
    with pytest.raises(KeyError):
        call(lib, "sgemm_fp4", format_="fp8")
    with pytest.raises(KeyError):
        call(lib, "sgemm_experts_layer", wtype="fp4")
