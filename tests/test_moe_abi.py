"""Refusals of the calls for experts and adapters: status codes of the C entries
(before any CUDA call, so no device is needed) and the Python binding's checks."""

import pytest
import torch

from fp4_fp8_quant_gb300 import build as B

ARG, ALIGN, SHAPE, WORKSPACE = -1, -2, -3, -6
ENOUGH = 1 << 40


@pytest.fixture(scope="module")
def iq():
    B.build()
    from fp4_fp8_quant_gb300 import iq
    iq.lib()
    return iq


def _refusals(call, good, bad):
    for kw, want in bad:
        assert call(**(good | kw)) == want, kw


def test_quantised_rows(iq):
    f = iq.lib().iq_fp8_quant_1x128_rows

    def call(x, src, rows, M, K, ldx, y, ldy, s):
        return f(x, src, rows, M, K, ldx, y, ldy, s, None)

    good = dict(x=16, src=3, rows=4, M=4, K=256, ldx=256, y=16, ldy=256, s=4)
    _refusals(call, good, [
        (dict(M=-1), ARG), (dict(src=-1), ARG), (dict(K=0), SHAPE), (dict(K=200), SHAPE), (dict(x=None), ARG),
        (dict(rows=None), ARG), (dict(y=None), ARG), (dict(s=None), ARG), (dict(ldx=128), ARG), (dict(ldy=255), ARG),
        (dict(x=8), ALIGN), (dict(rows=2), ALIGN), (dict(y=24), ALIGN), (dict(s=6), ALIGN), (dict(ldx=260), ALIGN),
        (dict(ldy=264), ALIGN), (dict(M=0, x=None), 0), (dict(M=0, K=100), SHAPE)])


def test_route(iq):
    f = iq.lib().iq_moe_route

    def call(l, b, ld, T, E, k, score, norm, scale, w, e, s, r, st, ws, n):
        return f(l, b, ld, T, E, k, score, norm, scale, w, e, s, r, st, ws, n, None)

    good = dict(l=4, b=0, ld=64, T=300, E=64, k=8, score=0, norm=0, scale=1.0, w=4, e=4, s=4, r=4, st=4, ws=256, n=ENOUGH)
    need = iq.moe_route_workspace_bytes(300, 64)
    assert need == (19 + 1) * 64 * 4 and iq.moe_route_workspace_bytes(128, 64) == 0 < iq.moe_route_workspace_bytes(129, 63) < need
    assert iq.moe_route_workspace_bytes(100, 0) == iq.moe_route_workspace_bytes(100, 1025) == iq.moe_route_workspace_bytes(-1, 8) == 0
    _refusals(call, good, [
        (dict(T=-1), ARG), (dict(score=2), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
        (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=4, k=5), SHAPE),
        (dict(l=None), ARG), (dict(w=None), ARG), (dict(e=None), ARG), (dict(s=None), ARG), (dict(r=None), ARG),
        (dict(st=None), ARG), (dict(T=0, st=None), ARG), (dict(ld=63), ARG), (dict(T=1 << 30), ARG), (dict(T=(1 << 31) - 32, E=1, k=1), ARG),
        (dict(l=6), ALIGN),
        (dict(b=1, l=3), ALIGN), (dict(w=2), ALIGN), (dict(e=2), ALIGN), (dict(s=1), ALIGN), (dict(r=5), ALIGN),
        (dict(st=2), ALIGN), (dict(ws=None), ARG), (dict(ws=128), ALIGN), (dict(n=need - 1), WORKSPACE)])


@pytest.mark.gpu
def test_quantised_rows_of_no_source(cuda_device):
    """A list over an empty tensor names no row: zeros throughout."""
    from fp4_fp8_quant_gb300 import iq
    y, s = iq.fp8_quant_1x128_ue8m0(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"),
                                    rows=torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda"))
    want, ws = iq.fp8_quant_1x128_ue8m0(torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(y, want) and torch.equal(s, ws)


def test_route_workspace_never_falls(iq):
    """A workspace for the most tokens and experts serves all calls of fewer."""
    size = iq.moe_route_workspace_bytes
    tokens = sorted([*range(1, 9000, 7), *range(2040, 2060), 1 << 20])
    for experts in (1, 64, 255, 256, 1024):
        bytes_ = [size(T, experts) for T in tokens]
        assert bytes_ == sorted(bytes_)
        assert all(size(T, experts) <= size(T, min(1024, experts + 1)) for T in (1, 129, 2048, 2049, 9000))


def test_grouped_gemm(iq):
    f = iq.lib().iq_grouped_gemm

    def call(x, ldx, xs, M, K, w, sf, G, N, st, g, y, ldy, ws, n):
        return f(x, ldx, xs, M, K, w, sf, G, N, st, g, y, ldy, ws, n, None)

    good = dict(x=16, ldx=7168, xs=4, M=40, K=7168, w=16, sf=1, G=3, N=512, st=4, g=0, y=16, ldy=512, ws=256, n=ENOUGH)
    size = iq.grouped_gemm_workspace_bytes
    need = size(40, 7168)
    assert size(0, 7168) == size(-3, 7168) == size(40, 0) == size(40, 200) == size(40, 1 << 21) == size(40, 1536) == 0
    assert 0 < need < size(256, 7168) == size(1 << 20, 7168) < 1 << 26
    _refusals(call, good, [
        (dict(M=-1), ARG), (dict(K=0), SHAPE), (dict(K=500), SHAPE), (dict(K=1 << 21), SHAPE), (dict(G=0), SHAPE),
        (dict(G=1025), SHAPE), (dict(N=0), SHAPE), (dict(N=12), SHAPE), (dict(N=384, g=1), SHAPE), (dict(M=0, N=12), SHAPE),
        (dict(M=(1 << 31) - 1, G=1024), SHAPE), (dict(M=1 << 30, G=128), SHAPE), (dict(M=0, x=None, y=None, ws=None), 0), (dict(x=None), ARG),
        (dict(xs=None), ARG), (dict(w=None), ARG), (dict(sf=None), ARG), (dict(st=None), ARG), (dict(y=None), ARG),
        (dict(ldx=7152), ARG), (dict(ldy=504), ARG), (dict(g=1, ldy=248), ARG), (dict(x=24), ALIGN), (dict(ldx=7176), ALIGN),
        (dict(xs=2), ALIGN), (dict(w=8), ALIGN), (dict(st=6), ALIGN), (dict(y=8), ALIGN), (dict(ldy=516), ALIGN),
        (dict(ws=None), ARG), (dict(ws=64), ALIGN), (dict(n=need - 1), WORKSPACE), (dict(K=1536, ws=None, n=0, y=None), ARG)])


def test_grouped_gemm_workspace_never_falls(iq):
    """A workspace for the largest batch serves the smaller ones."""
    size = iq.grouped_gemm_workspace_bytes
    widths = [M for M in range(1, 300)] + [512, 4632, 1 << 20]
    for K in range(128, 8192, 128):
        bytes_ = [size(M, K) for M in widths]
        assert bytes_ == sorted(bytes_), K
        assert (bytes_[0] > 0) == (K > 2304) and all(a <= size(M, K + 128) for a, M in zip(bytes_, widths))


def test_combine(iq):
    f = iq.lib().iq_moe_combine

    def call(y, ldy, S, sl, w, T, k, N, a, lda, o, ldo):
        return f(y, ldy, S, sl, w, T, k, N, a, lda, o, ldo, None)

    good = dict(y=16, ldy=64, S=9, sl=4, w=4, T=3, k=2, N=64, a=None, lda=0, o=16, ldo=64)
    _refusals(call, good, [
        (dict(T=-1), ARG), (dict(S=-1), ARG), (dict(N=0), SHAPE), (dict(N=60), SHAPE), (dict(k=0), SHAPE),
        (dict(T=0, y=None, o=None), 0), (dict(T=0, N=60), SHAPE), (dict(sl=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG),
        (dict(o=None), ARG), (dict(ldy=56), ARG), (dict(ldo=56), ARG), (dict(a=16, lda=56), ARG), (dict(sl=2), ALIGN),
        (dict(w=1), ALIGN), (dict(y=8), ALIGN), (dict(o=18), ALIGN), (dict(a=4, lda=64), ALIGN), (dict(ldy=68), ALIGN)])


def test_adapters(iq):
    f = iq.lib().iq_adapters

    def call(x, ldx, T, K, a, b, sc, A, r, N, st, ad, R, ba, ldb, o, ldo, ws, n):
        return f(x, ldx, T, K, a, b, sc, A, r, N, st, ad, R, ba, ldb, o, ldo, ws, n, None)

    good = dict(x=16, ldx=64, T=9, K=64, a=16, b=16, sc=4, A=2, r=16, N=64, st=4, ad=4, R=3, ba=16, ldb=64, o=16, ldo=64, ws=256,
                n=ENOUGH)
    need = iq.adapters_workspace_bytes(9, 16)
    assert need > 0 and iq.adapters_workspace_bytes(0, 16) == iq.adapters_workspace_bytes(9, 12) == 0
    assert iq.adapters_workspace_bytes(9, 136) == iq.adapters_workspace_bytes(9, 0) == iq.adapters_workspace_bytes(-9, 16) == 0
    _refusals(call, good, [
        (dict(T=-1), ARG), (dict(R=-1), ARG), (dict(K=0), SHAPE), (dict(K=60), SHAPE), (dict(N=0), SHAPE), (dict(N=66), SHAPE),
        (dict(r=0), SHAPE), (dict(r=12), SHAPE), (dict(r=136), SHAPE), (dict(A=0), SHAPE), (dict(R=1025), SHAPE),
        (dict(T=1 << 30, N=1 << 16), SHAPE), (dict(T=1 << 29), SHAPE), (dict(T=0, x=None), 0), (dict(R=0, x=None), 0), (dict(x=None), ARG),
        (dict(a=None), ARG), (dict(b=None), ARG), (dict(sc=None), ARG), (dict(st=None), ARG), (dict(ad=None), ARG),
        (dict(o=None), ARG), (dict(ldx=56), ARG), (dict(ldb=56), ARG), (dict(ldo=0), ARG), (dict(x=8), ALIGN), (dict(a=8), ALIGN),
        (dict(b=4), ALIGN), (dict(sc=2), ALIGN), (dict(st=1), ALIGN), (dict(ad=2), ALIGN), (dict(ba=8), ALIGN), (dict(o=8), ALIGN),
        (dict(ldx=68), ALIGN), (dict(ldb=65), ALIGN), (dict(ldo=66), ALIGN), (dict(ws=None), ARG), (dict(ws=8), ALIGN),
        (dict(n=need - 1), WORKSPACE)])


def test_cpu_tensors_never_reach_the_library(iq):
    bf, i32, u8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
    z = lambda *s, t=bf: torch.zeros(s, dtype=t)
    with pytest.raises(ValueError, match="CUDA"):
        iq.moe_route(z(4, 8, t=f32), 2)
    with pytest.raises(ValueError, match="CUDA"):
        iq.fp8_quant_1x128_ue8m0(z(4, 128), rows=z(4, t=i32))
    with pytest.raises(ValueError, match="CUDA"):
        iq.grouped_gemm(z(4, 128, t=u8), z(1, 4, t=i32), z(1, 128, 128, t=u8), z(1, 1, 1, t=u8), z(2, t=i32))
    with pytest.raises(ValueError, match="CUDA"):
        iq.moe_combine(z(4, 64), z(2, 2, t=i32), z(2, 2, t=f32))
    with pytest.raises(ValueError, match="CUDA"):
        iq.adapters(z(4, 64), None, z(1, 8, 64), z(1, 64, 8), z(1, t=f32), z(2, t=i32), z(1, t=i32))
    with pytest.raises(ValueError, match="score"):
        iq.moe_route(z(4, 8, t=f32), 2, score="other")


def test_another_gpu_than_the_current_one_is_refused(iq, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    elsewhere = type("T", (), {"is_cuda": True, "device": torch.device("cuda", 1)})
    with pytest.raises(ValueError, match="not the current GPU"):
        iq._check_device(elsewhere, "x")
    with pytest.raises(ValueError, match="CUDA"):
        iq._check_device(torch.zeros(1), "x")


def test_sizes_at_the_end_of_32_bits(iq):
    """Sizes that no longer fit 32 bits once they are rounded up to tiles: refused, and
    counted before they are."""
    L, end = iq.lib(), (1 << 31) - 8
    wide = (1 << 31) - 128
    assert L.iq_fp8_quant_1x128_rows(16, 3, 4, 1, wide, wide, 16, wide, 4, None) == SHAPE
    assert L.iq_fp8_quant_1x128_rows(16, 3, 4, end, 128, 128, 16, 128, 4, None) == SHAPE
    for M, N in ((1, end), (end, 8)):
        assert L.iq_grouped_gemm(16, 128, 4, M, 128, 16, 1, 1, N, 4, 0, 16, N, 256, ENOUGH, None) == SHAPE
    for K, N in ((end, 8), (8, end)):                          # 2^25 steps of K, 2^24 tiles of features
        assert L.iq_adapters(16, K, 1, K, 16, 16, 4, 1, 8, N, 4, 4, 1, None, 0, 16, N, 256, 0, None) == SHAPE


def test_binding_fails_loudly_without_its_module(iq, tmp_path, monkeypatch):
    monkeypatch.setattr(iq, "_binding", None)
    monkeypatch.setattr(iq, "BINDING_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(ImportError):
        iq._load_binding()


def test_binding_of_another_pytorch_or_python_is_not_taken(iq, monkeypatch):
    """The module writes PyTorch's own structures, so it is found by the versions it
    was compiled for, and built again where they have changed."""
    import sysconfig
    name = iq.BINDING_PATH.rsplit("/", 1)[1]
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert B.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.1")
    assert B.binding_path() != iq.BINDING_PATH and not B.up_to_date()
    monkeypatch.setattr(iq, "_binding", None)
    monkeypatch.setattr(iq, "BINDING_PATH", B.binding_path())
    with pytest.raises(ImportError, match="not built for this PyTorch"):
        iq._load_binding()


@pytest.mark.gpu
def test_python_checks_on_gpu_tensors(cuda_device):
    from fp4_fp8_quant_gb300 import iq
    dev = "cuda"
    bf, i32, u8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
    z = lambda *s, t=bf: torch.zeros(s, dtype=t, device=dev)

    def refuses(f, good, bad, err=ValueError):
        f(**good)
        for kw in bad:
            with pytest.raises(err):
                f(**(good | kw))

    logits = z(5, 16, t=f32)
    refuses(iq.moe_route, dict(logits=logits, k=3),
            [dict(logits=logits.half()), dict(logits=logits[0]), dict(logits=logits.t().contiguous().t()), dict(k=0), dict(k=17),
             dict(logits=z(5, 40, t=f32), k=33), dict(workspace=z(64, t=f32)), dict(score="max")])
    with pytest.raises(iq.IQError):
        iq.moe_route(z(5, 1025, t=f32), 3)
    with pytest.raises(iq.IQError):
        iq.moe_route(z(300, 16, t=f32), 3, workspace=z(16, t=u8))

    x, rows = z(5, 256), z(7, t=i32)
    refuses(lambda x, rows, y=None, scales=None: iq.fp8_quant_1x128_ue8m0(x, y, scales, rows=rows), dict(x=x, rows=rows),
            [dict(x=x.float()), dict(x=x[0]), dict(rows=rows.long()), dict(rows=rows[None]), dict(rows=rows.cpu()),
             dict(rows=z(14, t=i32)[::2]), dict(y=z(7, 128, t=u8)), dict(y=z(7, 256)), dict(scales=z(1, 7, t=i32))])
    with pytest.raises(iq.IQError):
        iq.fp8_quant_1x128_ue8m0(z(5, 200), rows=rows)

    q, s, w, sf, st = z(7, 4096, t=u8), z(8, 8, t=i32), z(2, 512, 4096, t=u8), z(2, 4, 32, t=u8), z(3, t=i32)
    good = dict(x=q, x_scales=s, w=w, w_sf=sf, row_start=st)
    refuses(iq.grouped_gemm, good,
            [dict(x=q.int()), dict(x=q[0]), dict(x_scales=s[:, :7]), dict(x_scales=s.float()), dict(w=w[0]), dict(w=w[:, :, :128]),
             dict(w=w.transpose(0, 1)), dict(w_sf=sf[:, :3]), dict(w_sf=sf.int()), dict(row_start=st[:2]), dict(row_start=st.cpu()),
             dict(out=z(7, 511)), dict(out=z(7, 512, t=f32)), dict(gated=True, out=z(7, 512)), dict(workspace=z(9, t=f32))])
    for kw in (dict(workspace=z(16, t=u8)), dict(w=z(2, 384, 4096, t=u8), w_sf=z(2, 3, 32, t=u8), gated=True), dict(out=z(7, 516)[:, :512])):
        with pytest.raises(iq.IQError):
            iq.grouped_gemm(**(good | kw))

    y, slots, wt = z(6, 64), z(3, 2, t=i32), z(3, 2, t=f32)
    refuses(iq.moe_combine, dict(y=y, slots=slots, weights=wt),
            [dict(y=y.float()), dict(y=y[0]), dict(slots=slots.long()), dict(slots=slots[0]), dict(weights=wt[:2]),
             dict(weights=wt.double()), dict(add=y), dict(add=z(3, 64, t=f32)), dict(out=z(3, 72)), dict(add=z(3, 64).cpu())])
    with pytest.raises(iq.IQError):
        iq.moe_combine(z(6, 60), slots, wt)

    good = dict(x=z(4, 64), base=z(4, 72), a=z(2, 8, 64), b=z(2, 72, 8), scale=z(2, t=f32), row_start=z(4, t=i32), adapter=z(3, t=i32))
    refuses(iq.adapters, good,
            [dict(x=z(4, 64, t=f32)), dict(x=z(4, 72)), dict(base=z(4, 64)), dict(base=z(3, 72)), dict(a=z(2, 8, 72)), dict(a=z(8, 64)),
             dict(b=z(2, 72, 16)), dict(b=z(3, 72, 8)), dict(scale=z(3, t=f32)), dict(scale=z(2)), dict(row_start=z(3, t=i32)),
             dict(row_start=z(4, t=torch.int64)), dict(adapter=z(3)), dict(out=z(4, 64)), dict(workspace=z(9))])
    with pytest.raises(iq.IQError):
        iq.adapters(**(good | dict(a=z(2, 12, 64), b=z(2, 72, 12))))
    with pytest.raises(iq.IQError):
        iq.adapters(**(good | dict(workspace=z(16, t=u8))))
    torch.cuda.synchronize()
