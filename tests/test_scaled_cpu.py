"""Block-scaled 8-bit layers on a host without a GPU: what the C entry points refuse before any launch, their workspaces,
and the compiled kernels' matrix-core wait states."""
import ctypes
import os
import tempfile

import pytest

import isa_waitstates as isa
import tile_gemm_amd as hts
from tile_gemm_amd import build as hb

A16, A8, A4, A2 = 0x10000, 0x10008, 0x10004, 0x10002   # never dereferenced: every call fails its host checks
by = ctypes.byref


def weight(**k):
    d = dict(values=A16, ld=512, scale=A4, ld_scale=4)
    d.update(k)
    return hts.hts_scaled_weight(*d.values())


def quant(entry="rows", **k):
    a = dict(dtype=hts.HTS_BF16, M=8, K=512, X=A16, ldx=512, Q=A16, ldq=512, scale=A4, lds=8)
    a.update(k)
    f = hts.lib().hts_quantize_rows if entry == "rows" else hts.lib().hts_quantize_weight
    return f(*a.values(), None)


def gemm(w=None, **k):
    a = dict(M=8, N=300, K=512, X=A16, ldx=512, xs=A4, ldxs=8, W=by(w or weight()), Y=A16, ldy=300, yd=hts.HTS_BF16,
             ws=None, nb=0)
    a.update(k)
    return hts.lib().hts_scaled_gemm(*a.values(), None)


def gated(w=None, u=None, **k):
    a = dict(act=0, M=8, N=304, K=512, X=A16, ldx=512, xs=A4, ldxs=8, G=by(w or weight()), U=by(u or weight()), H=A16,
             ldh=304, hd=hts.HTS_F16, hs=None, ldhs=0, ws=None, nb=0)
    a.update(k)
    return hts.lib().hts_scaled_gated(*a.values(), None)


def mlp(w=None, u=None, d=None, **k):
    a = dict(act=0, dt=hts.HTS_BF16, M=8, hidden=512, inner=304, X=A16, ldx=512, G=by(w or weight()), U=by(u or weight()),
             D=by(d or weight(ld=304, ld_scale=3)), Y=A16, ldy=512, ws=A16, nb=1 << 30)
    a.update(k)
    return hts.lib().hts_scaled_mlp(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), 2), (dict(dtype=7), 2), (dict(M=-1), 3), (dict(K=0), 3), (dict(K=-16), 3), (dict(K=24, ldx=24, ldq=32), 3),
    (dict(K=1 << 22, ldx=1 << 22, ldq=1 << 22), 7), (dict(M=1 << 26), 7), (dict(X=None), 1), (dict(X=A8), 4), (dict(ldx=504), 3),
    (dict(ldx=516), 4), (dict(Q=None), 1), (dict(Q=A8), 4), (dict(ldq=496), 3), (dict(ldq=520), 4), (dict(scale=None), 1),
    (dict(scale=A2), 4), (dict(lds=1 << 31), 3),
])
def test_quantisers_refuse(change, status):
    for entry in ("rows", "weight"):
        assert quant(entry, **change) == status, (entry, hts.lib().hts_last_error())


def test_quantiser_scale_layouts():
    assert quant("rows", lds=7) == 3 and quant("weight", lds=3) == 3
    assert quant("rows", M=0, X=None, Q=None, scale=None) == 0


COMMON = [
    (dict(M=-1), 3), (dict(N=0), 3), (dict(K=0), 3), (dict(K=500), 3), (dict(K=1 << 22), 7), (dict(M=1 << 26), 7),
    (dict(N=1 << 26), 7), (dict(X=None), 1), (dict(X=A8), 4), (dict(ldx=496), 3), (dict(ldx=520), 4), (dict(ldx=1 << 22), 7),
    (dict(xs=None), 1), (dict(xs=A2), 4), (dict(ldxs=7), 3), (dict(ws=A8, nb=64), 4),
]


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(W=None), 1), (dict(Y=None), 1), (dict(Y=A8), 4), (dict(ldy=299), 3), (dict(ldy=302), 4), (dict(yd=3), 2), (dict(yd=9), 2),
])
def test_product_refuses(change, status):
    assert gemm(**change) == status, hts.lib().hts_last_error()


BAD_WEIGHTS = [(dict(values=None), 1), (dict(values=A8), 4), (dict(ld=496), 3), (dict(ld=520), 4), (dict(ld=1 << 22), 7),
               (dict(scale=None), 1), (dict(scale=A2), 4), (dict(ld_scale=3), 3)]


@pytest.mark.parametrize("change,status", BAD_WEIGHTS)
def test_weights_are_refused(change, status):
    w = weight(**change)
    assert gemm(w) == status and gated(w) == status and gated(None, w) == status and mlp(w) == status and mlp(None, w) == status


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(act=-1), 1), (dict(act=3), 1), (dict(G=None), 1), (dict(U=None), 1), (dict(H=None), 1), (dict(H=A8), 4), (dict(ldh=300), 3),
    (dict(ldh=306), 4), (dict(hd=4), 2), (dict(hs=A16, ldhs=8), 1),
    (dict(hd=3), 1), (dict(hd=3, hs=A2, ldhs=8), 4), (dict(hd=3, hs=A4, ldhs=7), 3), (dict(hd=3, hs=A4, ldhs=8, ldh=312), 4),
    (dict(hd=3, hs=A4, ldhs=8, N=300), 3), (dict(hd=3, hs=A4, ldhs=8), 6), (dict(hd=3, hs=A4, ldhs=8, ws=A16, nb=64), 6),
])
def test_gated_refuses(change, status):
    assert gated(**change) == status, hts.lib().hts_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(act=5), 1), (dict(dt=2), 2), (dict(dt=3), 2), (dict(M=-1), 3), (dict(hidden=0), 3), (dict(hidden=500), 3), (dict(inner=0), 3),
    (dict(inner=300), 3), (dict(X=None), 1), (dict(X=A8), 4), (dict(ldx=504), 3), (dict(ldx=516), 4), (dict(G=None), 1), (dict(U=None), 1),
    (dict(D=None), 1), (dict(Y=None), 1), (dict(Y=A2), 4), (dict(ldy=508), 3), (dict(ws=None), 1), (dict(ws=A8), 4), (dict(nb=16), 6),
    (dict(ldx=520, ldy=512), 1),
])
def test_mlp_refuses(change, status):
    assert mlp(**change) == status, hts.lib().hts_last_error()


def test_nothing_to_do():
    assert gemm(M=0, X=None, Y=None) == 0 and gated(M=0, X=None) == 0 and mlp(M=0, X=None, ws=None, nb=0) == 0


def test_workspaces():
    n = ctypes.c_size_t(0)
    L = hts.lib()
    assert L.hts_scaled_gemm_workspace(8, 300, 500, by(n)) == 3 and L.hts_scaled_gemm_workspace(8, 300, 512, None) == 1
    assert L.hts_scaled_gated_workspace(8, 300, 512, 5, by(n)) == 2 and L.hts_scaled_mlp_workspace(8, 512, 300, by(n)) == 3
    assert hts.hts_scaled_gemm_workspace(0, 4096, 4096) == 0
    # E4M3 rows of a small batch go through 32-bit sums of gate and up
    assert hts.hts_scaled_gated_workspace(8, 304, 512, "fp8") >= 2 * 8 * 304 * 4


SOURCES = ["scaled_stream.hip", "scaled_ring.hip", "scaled_tile.hip"]
OP = "v_mfma_f32_16x16x128_f8f6f4"


@pytest.fixture(scope="module")
def need():
    try:
        hipcc = hb.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    flags = [f for f in hb.COMMON if f != "-fPIC"] + hb.VGPR_FORM
    with pytest.MonkeyPatch.context() as m:
        m.setitem(isa.PROBE_OPS, OP,
                  "acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(I8[l], I8[l + 64], acc, 0, 0, 0, 0, 0, 0);")
        w = isa.required_waits(flags, hipcc)
    assert w[OP] == w["v_mfma_scale_f32_16x16x128_f8f6f4"]
    return w, flags, hipcc


@pytest.mark.parametrize("src", SOURCES)
def test_scaled_kernels_respect_wait_states(need, src):
    w, flags, hipcc = need
    with tempfile.TemporaryDirectory() as d:
        text = isa.device_asm(os.path.join(hb.CSRC, src), os.path.join(d, "k.s"), flags, hipcc)
    assert OP in text
    bad = isa.violations(text, w)
    assert not bad, f"{len(bad)} early reads, first: {bad[:3]}"
