"""The steps around the products on a host without a GPU: what they refuse, before any launch, and the
rotary plan against extended precision."""
import ctypes
import re

import numpy as np
import pytest
import torch

import serving_ref as ref
import tile_gemm_amd as hts

A16, A8, A4, A2 = 0x10000, 0x10008, 0x10004, 0x10002   # never dereferenced: every call fails its host checks
by = ctypes.byref


def kv(**k):
    d = dict(pages=64, page=16, heads=8, dim=128, dtype=hts.HTS_BF16, page_stride=16 * 8 * 128,
             token_stride=8 * 128, head_stride=128)
    d.update(k)
    return hts.hts_kv_desc(**d)


# ---- page step -------------------------------------------------------------

def step(**k):
    a = dict(B=4, cached=0x100000, added=0x200000, page=16, free=0x300000, n_free=100, head=0x400000, table=0x500000,
             ldt=8, width=8, tokens=32, lengths=0x600000, starts=0x700000, slots=0x800000, positions=0x900000,
             head_out=0xA00000)
    a.update(k)
    return hts.lib().hts_kv_step(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), 3), (dict(B=4097), 7), (dict(page=8), 7), (dict(page=24), 7), (dict(page=2048), 7), (dict(page=0), 7),
    (dict(page=-16), 7), (dict(cached=None), 1), (dict(added=None), 1), (dict(free=None), 1), (dict(table=None), 1),
    (dict(lengths=None), 1), (dict(starts=None), 1), (dict(slots=None), 1), (dict(positions=None), 1),
    (dict(head_out=None), 1), (dict(cached=0x100002), 4), (dict(slots=0x800004), 4), (dict(head=0x400001), 4),
    (dict(ldt=7), 3), (dict(width=0), 3), (dict(ldt=2 ** 31), 3), (dict(tokens=-1), 3), (dict(tokens=2 ** 31), 3),
    (dict(n_free=-1), 3), (dict(B=4096, width=2 ** 19, ldt=2 ** 19), 3),
    (dict(lengths=0x100000), 1), (dict(head_out=0x400000), 1), (dict(lengths=0x100000 - 12), 1),
    (dict(positions=0x700010), 1), (dict(table=0x300000), 1), (dict(slots=0x500008), 1),
])
def test_step_refuses(change, status):
    assert step(**change) == status, hts.lib().hts_last_error()


# ---- rotary ----------------------------------------------------------------

def rope_desc(**k):
    d = dict(dtype=hts.HTS_BF16, layout=0, dim=128, rot=128, q_heads=32, k_heads=8, magnitude=1.0, reserved=0)
    d.update(k)
    return hts.hts_rope_desc(**d)


def rope(desc=None, **k):
    a = dict(turns=A16, T=4, positions=A16, Q=A16, ldq=4096, Qo=A16, ldqo=4096, K=A16, ldk=1024, Ko=A16, ldko=1024)
    a.update(k)
    return hts.lib().hts_rope(by(desc or rope_desc()), *a.values(), None)


def rope_cache(desc=None, cache=None, **k):
    a = dict(turns=A16, T=4, positions=A16, slots=A16, Q=A16, ldq=4096, Qo=A16, ldqo=4096, K=A16, ldk=1024, V=A16,
             ldv=1024, kv=by(cache or kv()), kc=0x100000, vc=0x200000, ks=None, vs=None)
    a.update(k)
    return hts.lib().hts_rope_cache(by(desc or rope_desc()), *a.values(), None)


def test_rope_refuses():
    assert hts.lib().hts_rope(None, A16, 4, A16, A16, 4096, A16, 4096, A16, 1024, A16, 1024, None) == 1
    for change, status in ((dict(dtype=2), 2), (dict(dtype=3), 2), (dict(layout=2), 1), (dict(dim=12), 7),
                           (dict(dim=264, rot=8), 7), (dict(rot=0), 7), (dict(rot=12), 7), (dict(rot=136), 7),
                           (dict(q_heads=-1), 3), (dict(reserved=1), 1), (dict(magnitude=float("inf")), 1)):
        assert rope(rope_desc(**change)) == status, change
        assert rope_cache(rope_desc(**change)) == status, change
    for change, status in ((dict(T=-1), 3), (dict(T=2 ** 31), 3), (dict(turns=None), 1), (dict(turns=A4), 4),
                           (dict(positions=None), 1), (dict(positions=A2), 4), (dict(Q=None), 1), (dict(Q=A8), 4),
                           (dict(ldq=4088), 3), (dict(ldq=4100), 4), (dict(Qo=None), 1), (dict(ldqo=4104), 1)):
        assert rope(**change) == status, change
        assert rope_cache(**change) == status, change
    assert rope(K=None) == 1 and rope(Ko=A8) == 4 and rope(ldko=1032) == 1 and rope(ldk=1000) == 3
    assert rope(T=0, Q=None, turns=None) == 0
    assert rope(rope_desc(q_heads=0, k_heads=0), Q=None) == 0
    for change, status in ((dict(slots=None), 1), (dict(slots=A4), 4), (dict(V=None), 1), (dict(ldv=1020), 3),
                           (dict(kc=None), 1), (dict(vc=A8), 4), (dict(vc=0x100000), 1), (dict(kv=None), 1),
                           (dict(ks=A16), 1)):
        assert rope_cache(**change) == status, change
    assert rope_cache(cache=kv(heads=4)) == 3              # another number of heads
    assert rope_cache(cache=kv(dim=64)) == 3               # another head size
    assert rope_cache(cache=kv(dtype=hts.HTS_F16)) == 2    # another 16-bit type
    assert rope_cache(cache=kv(dtype=hts.HTS_FP8_E4M3), ks=A2) == 4
    assert rope_cache(T=0, slots=None, kc=None) == 0


def test_rope_cache_rows_refuses():
    def rows(desc=None, cache=None, **k):
        a = dict(turns=A16, B=4, starts=A16, tokens=4, positions=A16, slots=A16, Q=A16, ldq=4096, Qo=A16, ldqo=4096, K=A16,
                 ldk=1024, V=A16, ldv=1024, kv=by(cache or kv()), kc=0x100000, vc=0x200000, ks=None, vs=None)
        a.update(k)
        return hts.lib().hts_rope_cache_rows(by(desc or rope_desc()), *a.values(), None)
    for change, status in ((dict(B=-1), 3), (dict(B=2 ** 31), 3), (dict(starts=None), 1), (dict(starts=A2), 4), (dict(tokens=0), 3),
                           (dict(tokens=-1), 3), (dict(tokens=2 ** 31), 3), (dict(positions=None), 1), (dict(slots=A4), 4),
                           (dict(Q=None), 1), (dict(ldqo=4104), 1), (dict(V=None), 1), (dict(vc=0x100000), 1), (dict(kv=None), 1)):
        assert rows(**change) == status, change
    assert rows(rope_desc(rot=12)) == 7 and rows(cache=kv(heads=4)) == 3
    assert rows(B=0, tokens=0, starts=None, positions=None, slots=None, kc=None) == 0


@pytest.mark.parametrize("change,status", [
    (dict(pages=0), 3), (dict(pages=2 ** 31), 3), (dict(page=8), 7), (dict(page=48), 7), (dict(heads=0), 3),
    (dict(dim=4), 7), (dict(dim=260), 7), (dict(dtype=hts.HTS_F32), 2), (dict(dtype=9), 2), (dict(head_stride=0), 3),
    (dict(head_stride=-128), 3), (dict(head_stride=132), 4), (dict(head_stride=120), 3), (dict(token_stride=1016), 3),
    (dict(page_stride=16 * 1024 - 8), 3), (dict(page_stride=2 ** 48), 3),
    (dict(page_stride=1024, token_stride=1024), 3), (dict(pages=2 ** 31 - 1, page_stride=2 ** 47), 3),
])
def test_cache_descriptions_that_are_refused(change, status):
    n = ctypes.c_size_t(0)
    assert hts.lib().hts_paged_attn_workspace(4, 32, by(kv(**change)), 8, 0, by(n)) == status


def test_cache_descriptions_that_are_taken():
    n = ctypes.c_size_t(0)
    for change in (dict(), dict(token_stride=128, head_stride=16 * 128),           # heads outside the page's tokens
                   dict(pages=1, page_stride=0), dict(heads=1, head_stride=3),      # strides of single entries
                   dict(head_stride=64 * 16 * 128, token_stride=128, page_stride=16 * 128),   # heads outermost
                   dict(dtype=hts.HTS_FP8_E4M3, dim=8, head_stride=8, token_stride=64, page_stride=1024)):
        assert hts.lib().hts_paged_attn_workspace(4, 32, by(kv(**change)), 8, 0, by(n)) == 0, change


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [hts.HTS_BF16, hts.HTS_FP8_E4M3])
def test_unused_strides_change_nothing(dim, dtype):
    # one cache head, or one page: whatever stands in that axis's stride, the same memory is divided alike
    def bytes_of(**change):
        d = kv(**{**dict(heads=1, dim=dim, dtype=dtype, token_stride=dim, page_stride=16 * dim, head_stride=dim), **change})
        return hts.hts_paged_attn_workspace(64, 16, d, 512)
    assert bytes_of() > 0
    assert len({bytes_of(head_stride=s) for s in (dim, 16 * dim, 0, -8, 3, 2 ** 40)}) == 1
    assert len({bytes_of(pages=1, page_stride=s) for s in (16 * dim, 0, -8, 3, 2 ** 40)}) == 1


@pytest.mark.parametrize("rule,factor,context", [("plain", 1.0, 0.0), ("plain", 3.0, 0.0), ("linear", 4.0, 0.0), ("base", 8.0, 0.0),
                                                 ("ramp", 8.0, 4096.0), ("ramp_pairs", 16.0, 4096.0),
                                                 ("ramp_pairs", 2.5, 100.0)])
@pytest.mark.parametrize("rot", [8, 64, 128, 256])
@pytest.mark.parametrize("theta", [10000.0, 1e6])
def test_rope_plan(rule, factor, context, rot, theta):
    rules = {"plain": 0, "linear": 1, "base": 2, "ramp": 3, "ramp_pairs": 4}
    got = hts.hts_rope_plan(hts.hts_rope_scaling(rot, rules[rule], theta, factor, context, 1.0, 32.0))
    want = ref.rope_turns(rot, theta, rule, factor, context)
    # pow is within a few steps of 2^-53, its argument's rounding counts ln(theta) times more; "base" raises twice.
    # A ramp's c is a difference of numbers up to its slope's size: the same steps, times its turns (<= 652) / 31.
    assert np.all(np.abs(got - want) <= 2.0 ** -47 * np.abs(want).astype(np.float64))


def test_rope_plan_refuses():
    def plan(rot=128, rule=0, theta=10000.0, factor=1.0, context=4096.0, low=1.0, high=32.0):
        t = np.zeros(128)
        s = hts.hts_rope_scaling(rot, rule, theta, factor, context, low, high)
        return hts.lib().hts_rope_plan(by(s), t.ctypes.data)
    assert plan() == 0
    assert plan(rot=0) == 7 and plan(rot=12) == 7 and plan(rot=264) == 7
    for bad in (dict(rule=5), dict(rule=-1), dict(theta=1.0), dict(theta=float("nan")), dict(factor=0.5),
                dict(rule=1, factor=float("inf")), dict(rule=3, factor=2.0, context=0.0),
                dict(rule=3, factor=2.0, low=0.0), dict(rule=4, factor=2.0, high=1.0),
                dict(rule=2, rot=8, theta=1e300, factor=1e300)):
        assert plan(**bad) == 1, bad
    assert hts.lib().hts_rope_plan(None, None) == 1


# ---- attention -------------------------------------------------------------

def attn(cache=None, **k):
    a = dict(dtype=hts.HTS_BF16, B=4, heads=32, kv=by(cache or kv()), Q=A16, ldq=4096, kc=A16, vc=A16, ks=None, vs=None,
             table=A16, ldt=8, width=8, lengths=A16, scale=0.1, window=0, O=A16, ldo=4096, lse=None, ws=None, wsb=0)
    a.update(k)
    return hts.lib().hts_paged_attn(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 2), (dict(dtype=3), 2), (dict(dtype=0), 2), (dict(B=-1), 3), (dict(B=65536), 3), (dict(heads=0), 3),
    (dict(heads=12), 3), (dict(heads=65536 + 8), 3), (dict(Q=None), 1), (dict(Q=A8), 4), (dict(ldq=4088), 3),
    (dict(ldq=4100), 4), (dict(kc=None), 1), (dict(vc=A8), 4), (dict(ks=A16), 1), (dict(table=None), 1),
    (dict(table=A2), 4), (dict(width=0), 3), (dict(ldt=7), 3), (dict(lengths=None), 1), (dict(lengths=A2), 4),
    (dict(scale=float("nan")), 1), (dict(window=-1), 3), (dict(O=None), 1), (dict(ldo=4000), 3), (dict(ldo=4104), 1),
    (dict(lse=A2), 4), (dict(ws=A8, wsb=1 << 20), 4), (dict(kv=None), 1),
])
def test_attn_refuses(change, status):
    assert attn(**change) == status, hts.lib().hts_last_error()


def test_attn_of_nothing():
    assert attn(B=0, Q=None, O=None, table=None, lengths=None) == 0


# ---- norm ------------------------------------------------------------------

def norm(M=4, N=64, **k):
    d = dict(dtype=1, r_dtype=1, post=1, pre=1, post_eps=1e-6, pre_eps=1e-6, scale=1.0, gate_act=0)
    a = dict(block=0x10000, ldb=64, pw=None, pb=None, gate=None, ldg=0, R=0x20000, ldr=64, qw=None, qb=None,
             Ro=0x30000, ldro=64, Y=0x40000, ldy=64)
    for key, v in k.items():
        (d if key in d else a)[key] = v
    return hts.lib().hts_residual_norm(by(hts.hts_norm_desc(**d)), M, N, *a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), 2), (dict(dtype=3), 2), (dict(r_dtype=0), 2), (dict(r_dtype=3), 2), (dict(post=3), 1),
    (dict(pre=-1), 1), (dict(gate_act=3), 1), (dict(post_eps=-1.0), 1), (dict(pre_eps=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(M=-1), 3), (dict(M=2 ** 31), 3), (dict(N=0), 3), (dict(N=60), 3),
    (dict(N=32776), 7), (dict(block=None, R=None), 1), (dict(Ro=None, Y=None), 1), (dict(block=None), 1),
    (dict(block=None, post=0, gate=0x50000), 1), (dict(block=A8), 4), (dict(ldb=56), 3), (dict(ldb=68), 4),
    (dict(gate=A8), 4), (dict(gate=0x50000, ldg=8), 3), (dict(R=A8), 4), (dict(ldr=60), 3), (dict(Ro=A8), 4),
    (dict(ldro=0), 3), (dict(Y=A8), 4), (dict(ldy=68), 4), (dict(pw=A8), 4), (dict(qb=A8), 4), (dict(Y=0x30000), 1),
    (dict(Ro=0x20000, ldro=72), 1), (dict(Y=0x20000, ldy=72), 1), (dict(Y=0x20000, r_dtype=2), 1),
    (dict(Y=0x10000, ldy=72), 1), (dict(Ro=0x10000, r_dtype=2), 1), (dict(gate=0x50000, ldg=0, Y=0x50000), 1),
])
def test_norm_refuses(change, status):
    assert norm(**change) == status, hts.lib().hts_last_error()


def test_norm_of_nothing():
    assert norm(M=0, block=None, R=None) == 0


# ---- tensor-level checks ---------------------------------------------------

def test_helpers_refuse_host_tensors_and_wrong_shapes():
    cpu = torch.zeros(4, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(hts.HTSError, match="GPU"):
        hts.residual_norm(cpu, cpu, pre=hts.Norm("rms"))
    with pytest.raises(hts.HTSError, match="GPU"):
        hts.kv_step(i32, i32, i32, i32.view(4, 1), 16, 4)
    with pytest.raises(hts.HTSError, match="GPU"):
        hts.rope(cpu, None, i32, hts.RopePlan(torch.zeros(64, dtype=torch.float64), 0, 128, 128, 1.0))
    with pytest.raises(hts.HTSError, match="GPU"):
        hts.KVCache(torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16), torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16))
    with pytest.raises(hts.HTSError):
        hts.residual_norm(None, None)
    with pytest.raises(hts.HTSError):
        hts.residual_norm(cpu[0], None)
    with pytest.raises(hts.HTSError):
        hts.rope_plan(64, rot=128, device="cpu")
    with pytest.raises(hts.HTSError):
        hts.rope_plan(64, layout="both", device="cpu")
    with pytest.raises(hts.HTSError):
        hts.KVCache(torch.zeros(4, 16, 1, 128), torch.zeros(4, 16, 1, 128))


# ---- compiled code ---------------------------------------------------------

def test_attention_kernels_respect_wait_states(tmp_path):
    # no matrix-core result is read before its wait states on any path of the compiled kernels
    import os
    from tile_gemm_amd import build as hb
    from isa_waitstates import device_asm, required_waits, violations
    try:
        hipcc = hb.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    flags = [f for f in hb.COMMON if f != "-fPIC"] + hb.VGPR_FORM
    text = device_asm(os.path.join(hb.CSRC, "attn_decode.hip"), str(tmp_path / "k.s"), flags, hipcc)
    assert "v_mfma_f32_16x16x32_bf16" in text
    # Two instructions of one kind land in the order of their issue: a later one may overwrite a part of the first's
    # result (one that nothing reads any more), or take exactly that result as its accumulator (chained by the
    # hardware); it may not read it as an operand, nor a part of it as its accumulator.
    def regs(x):
        lo, _, hi = x.strip("v[]").partition(":")
        return set(range(int(lo), int(hi or lo) + 1))

    def in_order(first, second):
        (op, out, *_), (op2, _, x, y, acc) = (re.split(r",? ", i)[:5] for i in (first, second))
        r = regs(out)
        return op == op2 and not (regs(x) | regs(y)) & r and (regs(acc) == r or not regs(acc) & r)
    bad = [x for x in violations(text, required_waits(flags, hipcc)) if not (x[2].startswith("v_mfma") and in_order(x[1], x[2]))]
    assert not bad, f"{len(bad)} early reads, first: {bad[:3]}"


def test_shorter_products_respect_wait_states(tmp_path, monkeypatch):
    # the products over 16 tokens, as producers, and any accumulator that passes between products of two kinds
    import os
    import isa_waitstates as iw
    from tile_gemm_amd import build as hb
    try:
        hipcc = hb.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    monkeypatch.setattr(iw, "_PROBE_HEAD", iw._PROBE_HEAD + "typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));\n")
    monkeypatch.setattr(iw, "PROBE_OPS", {
        "v_mfma_f32_16x16x16_f16": "const f16x4* q = (const f16x4*)H8; "
                                   "acc = __builtin_amdgcn_mfma_f32_16x16x16f16(q[l], q[l + 64], acc, 0, 0, 0);"})
    flags = [f for f in hb.COMMON if f != "-fPIC"] + hb.VGPR_FORM
    text = iw.device_asm(os.path.join(hb.CSRC, "attn_decode.hip"), str(tmp_path / "k.s"), flags, hipcc)
    need = iw.required_waits(flags, hipcc)
    assert need["v_mfma_f32_16x16x16_f16"] > 1 and "v_mfma_f32_16x16x16_f16" in text
    # of one kind results land in the order of issue: a product may write registers that an earlier one wrote
    late = [x for x in iw.violations(text, need) if x[2].split()[0] != x[1].split()[0]]
    assert not late, late[:3]
    same = [x for x in iw.violations(text, need) if x[2].split()[0] == x[1].split()[0]]
    for _, first, second in same:
        out = iw._regs(iw._ops(first)[1][0])
        _, a, b, acc = iw._ops(second)[1][:4]
        assert not out & (iw._regs(a) | iw._regs(b)) and (iw._regs(acc) == out or not iw._regs(acc) & out), (first, second)


def test_wide_grids_fit_their_axes(tmp_path):
    # workgroups of a launch in two axes: every one of n is there, an axis holds fewer than 2^32 threads of 1024 a group
    import os
    import subprocess
    from tile_gemm_amd import build as hb
    try:
        hipcc = hb.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    src = tmp_path / "grid.cpp"
    src.write_text("""#include <cstdio>
#include "serve_internal.h"
int main() {
    for (long long n : {1ll, 255ll, (1ll << 21) - 1, 1ll << 21, (1ll << 21) + 1, 1ll << 24, (1ll << 31) - 1}) {
        const hts::WideGrid w = hts::wide_grid(n);
        const long long x = w.x, rest = w.rest;
        const bool ok = x * 1024 < (1ll << 32) && rest <= 65535 && x * rest >= n && (rest - 1) * x < n && (rest == 1 || x == hts::kGridX);
        std::printf("%lld %s\\n", n, ok ? "ok" : "bad");
    }
}
""")
    flags = [f for f in hb.COMMON if f.startswith("-I") or f.startswith("-std")]
    subprocess.run([hipcc, *flags, "-x", "hip", f"--offload-arch={hb.ARCH}", "--cuda-host-only", "-c", str(src), "-o", str(tmp_path / "g.o")],
                   check=True, capture_output=True)
    subprocess.run([hipcc, str(tmp_path / "g.o"), "-o", str(tmp_path / "g")], check=True, capture_output=True)
    got = subprocess.run([str(tmp_path / "g")], capture_output=True, text=True, check=True).stdout.split()
    assert len(got) == 14 and set(got[1::2]) == {"ok"}, got
