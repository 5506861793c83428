"""Refusals of the MXFP4, expert-layer and block-norm calls that need no GPU: C argument checks (fake, misaligned
addresses that no call may reach) and the binding's tensor checks."""

import ctypes

import pytest
import torch

import weight_only_quantized_wq_amd as wq

from weight_only_quantized_wq_amd import _binding

BAD = 0x1001
OK = 0x2000
FAR = 0x10_0000_0000
lib = _binding.lib


def _fill(cls, defaults, kw):
    defaults.update(kw)
    assert set(defaults) == {n for n, _ in cls._fields_}
    return cls(**defaults)


def gemm(**kw):
    return _fill(wq.wq_gemm_mxfp4, dict(x=BAD, x_stride=64, xq=None, x_scale=None, q=OK, scale=OK, y_f32=FAR, y_bf16=None,
                                        y_stride=32, m=3, n=32, k=64), kw)


def moe(**kw):
    return _fill(wq.wq_moe_ffn, dict(x=BAD, x_stride=64, router=OK, logits=None, w13=OK, s13=OK, w2=OK, s2=OK, y_f32=FAR,
                                     y_bf16=None, y_stride=64, sel=None, gates=None, tokens=3, dim=64, f=32, e=8, top=2,
                                     format=8, renormalize=1), kw)


def norm(**kw):
    return _fill(wq.wq_block_norm, dict(h_f32=BAD, h_bf16=None, h_stride=64, out_f32=FAR, out_bf16=None, out_stride=64,
                                        f_f32=OK, f_bf16=None, f_stride=64, f_norm=OK, gate=OK, gate_stride=64, norm=OK,
                                        u=2 * FAR, u_stride=64, q=None, q_scale=None, rows=3, dim=64, scale=1.0, eps=1e-6,
                                        gate_kind=0), kw)


CALLS = {
    "gemm": (gemm, lambda d, p: lib.wq_gemm_mxfp4_prepare(ctypes.byref(d), OK, 1 << 40, ctypes.byref(p)),
             wq.wq_gemm_mxfp4_plan),
    "moe": (moe, lambda d, p: lib.wq_moe_ffn_prepare(ctypes.byref(d), OK, 1 << 40, ctypes.byref(p)), wq.wq_moe_ffn_plan),
    "norm": (norm, lambda d, p: lib.wq_block_norm_prepare(ctypes.byref(d), ctypes.byref(p)), wq.wq_block_norm_plan),
}


def status(call, **kw):
    make, prepare, plan = CALLS[call]
    return prepare(make(**kw), plan())


@pytest.mark.parametrize("call", CALLS)
def test_a_good_description_stops_only_at_its_misaligned_pointer(call):
    assert status(call) == 3
    assert "aligned" in wq.last_error()


@pytest.mark.parametrize("call,kw,rc", [
    ("gemm", dict(x=None), 1), ("gemm", dict(xq=OK), 1), ("gemm", dict(x=None, xq=OK), 1), ("gemm", dict(q=None), 1),
    ("gemm", dict(scale=None), 1), ("gemm", dict(y_f32=None), 1),
    ("gemm", dict(m=-1), 2), ("gemm", dict(m=(1 << 20) + 1), 2), ("gemm", dict(n=-1), 2), ("gemm", dict(n=(1 << 24) + 1), 2),
    ("gemm", dict(k=0), 2), ("gemm", dict(k=48), 2), ("gemm", dict(k=(1 << 18) + 32, x_stride=1 << 19), 2),
    ("gemm", dict(x_stride=56), 2), ("gemm", dict(x_stride=68), 2), ("gemm", dict(x_stride=(1 << 22) + 8), 2),
    ("gemm", dict(y_stride=31), 2), ("gemm", dict(x=OK, q=BAD), 3), ("gemm", dict(x=OK, scale=BAD), 3),
    ("gemm", dict(x=None, xq=OK, x_scale=OK + 2), 3), ("gemm", dict(x=OK, y_f32=FAR + 2), 3),
    ("gemm", dict(x=OK, y_f32=None, y_bf16=BAD), 3),
    ("moe", dict(x=None), 1), ("moe", dict(router=None), 1), ("moe", dict(logits=OK), 1), ("moe", dict(w13=None), 1),
    ("moe", dict(s13=None), 1), ("moe", dict(w2=None), 1), ("moe", dict(s2=None), 1), ("moe", dict(y_f32=None), 1),
    ("moe", dict(format=3), 2), ("moe", dict(format=0), 2), ("moe", dict(tokens=65), 2), ("moe", dict(tokens=-1), 2),
    ("moe", dict(dim=48, x_stride=48), 2), ("moe", dict(f=48), 2), ("moe", dict(dim=0), 2), ("moe", dict(f=0), 2),
    ("moe", dict(dim=32800, x_stride=32800, y_stride=32800), 2), ("moe", dict(f=32800), 2), ("moe", dict(e=0), 2),
    ("moe", dict(e=257), 2), ("moe", dict(top=0), 2), ("moe", dict(top=9), 2), ("moe", dict(e=20, top=17), 2),
    ("moe", dict(x_stride=56), 2), ("moe", dict(x_stride=68), 2), ("moe", dict(y_stride=63), 2),
    ("moe", dict(format=2, dim=40, x_stride=40), 2), ("moe", dict(x=OK, w13=BAD), 3), ("moe", dict(x=OK, w2=BAD), 3),
    ("moe", dict(x=OK, router=BAD), 3), ("moe", dict(x=OK, s13=OK + 2), 3), ("moe", dict(x=OK, s2=OK + 2), 3),
    ("moe", dict(x=OK, sel=BAD), 3), ("moe", dict(x=OK, gates=BAD), 3), ("moe", dict(x=OK, router=None, logits=BAD), 3),
    ("norm", dict(h_f32=None), 1), ("norm", dict(h_bf16=OK), 1), ("norm", dict(f_bf16=OK), 1),
    ("norm", dict(f_f32=None), 1), ("norm", dict(f_f32=None, f_norm=None), 1), ("norm", dict(out_bf16=FAR), 1),
    ("norm", dict(q=OK), 1), ("norm", dict(q_scale=OK), 1), ("norm", dict(out_f32=None, u=None, norm=None), 1),
    ("norm", dict(u=None), 1), ("norm", dict(rows=-1), 2), ("norm", dict(rows=(1 << 24) + 1), 2),
    ("norm", dict(dim=60), 2), ("norm", dict(dim=0), 2), ("norm", dict(dim=32776), 2),
    ("norm", dict(dim=40, q=FAR, q_scale=3 * FAR), 2), ("norm", dict(gate_kind=3), 2), ("norm", dict(gate_kind=-1), 2),
    ("norm", dict(eps=-1.0), 2), ("norm", dict(eps=float("nan")), 2), ("norm", dict(eps=float("inf")), 2),
    ("norm", dict(scale=float("nan")), 2), ("norm", dict(scale=float("inf")), 2), ("norm", dict(h_stride=56), 2),
    ("norm", dict(f_stride=68), 2), ("norm", dict(out_stride=60), 2), ("norm", dict(u_stride=56), 2),
    ("norm", dict(gate_stride=8), 2), ("norm", dict(h_f32=OK, norm=BAD), 3), ("norm", dict(h_f32=OK, u=BAD), 3),
    ("norm", dict(h_f32=OK, q=BAD, q_scale=OK), 3),
], ids=str)
def test_refusals(call, kw, rc):
    assert status(call, **kw) == rc, wq.last_error()


# results on what is read, or on each other
MEET = [
    ("gemm", dict(x=OK, y_f32=OK + 256)),                                       # x: 3 rows of 128 bytes
    ("gemm", dict(x=None, xq=OK, x_scale=OK, y_f32=OK + 92)),                   # 3 rows of 32
    ("gemm", dict(x=None, xq=OK, x_scale=0x8000, y_f32=0x8004)),
    ("gemm", dict(x=OK, q=0x8000, y_f32=0x8000 + 1020)), ("gemm", dict(x=OK, scale=0x8000, y_f32=0x8000 + 60)),
    ("gemm", dict(x=OK, y_bf16=FAR + 380)),
    ("moe", dict(x=OK, y_f32=OK + 256)), ("moe", dict(x=OK, w13=0x8000, y_f32=0x8000 + 16380)),
    ("moe", dict(x=OK, w2=0x8000, y_f32=0x8000 + 8188)), ("moe", dict(x=OK, sel=FAR)), ("moe", dict(x=OK, gates=FAR + 764)),
    ("moe", dict(x=OK, router=0x8000, sel=0x8000)), ("moe", dict(x=OK, sel=0x8000, gates=0x8014)),
    ("moe", dict(x=OK, router=None, logits=0x8000, gates=0x8000 + 92)),
    ("norm", dict(h_f32=OK, out_f32=OK + 16)), ("norm", dict(h_f32=OK, out_f32=OK, out_stride=72)),
    ("norm", dict(h_f32=OK, u=OK)), ("norm", dict(h_f32=FAR, h_stride=72)), ("norm", dict(h_f32=0x8000, f_f32=FAR)),
    ("norm", dict(h_f32=0x8000, u=FAR)), ("norm", dict(h_f32=0x8000, gate=2 * FAR)),
    ("norm", dict(h_f32=0x8000, q=2 * FAR, q_scale=OK)), ("norm", dict(h_f32=0x8000, q=3 * FAR, q_scale=3 * FAR + 92)),
]


@pytest.mark.parametrize("call,kw", MEET, ids=str)
def test_results_must_not_lie_on_inputs_or_each_other(call, kw):
    assert status(call, **kw) == 2, wq.last_error()
    assert "overlap" in wq.last_error()


@pytest.mark.parametrize("call,kw", [
    ("norm", dict(h_f32=FAR)),                                                  # in place
    ("norm", dict(h_f32=OK, f_f32=0x8000, gate=0x9000, gate_stride=0)),
    ("gemm", dict(x=OK, y_f32=OK + 384, q=0x8000, scale=0x9000)),              # right behind x
    ("moe", dict(x=OK, format=2, sel=3 * FAR, gates=3 * FAR + 24)),
], ids=str)
def test_neighbours_are_no_overlap(call, kw):
    # a right call ends where the device is asked for
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert status(call, **kw) == 4, wq.last_error()


@pytest.mark.parametrize("kw,rc", [(dict(format=2, s13=OK + 2), 4), (dict(format=2, s2=OK + 6), 4), (dict(format=2, s13=BAD), 3),
                                   (dict(format=2, s2=BAD), 3), (dict(format=8, s2=OK + 2), 3)], ids=str)
def test_int8_scales_need_the_alignment_of_their_elements(kw, rc):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert status("moe", x=OK, **kw) == rc, wq.last_error()


def test_quantiser_refusals():
    q, d = lib.wq_quantize_mxfp4, lib.wq_dequantize_mxfp4
    assert q(None, None, 1, 32, OK, FAR, None) == 1 and q(OK, OK, 1, 32, FAR, FAR, None) == 1
    assert q(OK, None, 1, 32, None, FAR, None) == 1 and q(OK, None, 1, 32, FAR, None, None) == 1
    assert q(OK, None, -1, 32, FAR, 2 * FAR, None) == 2 and q(OK, None, 1, 40, FAR, 2 * FAR, None) == 2
    assert q(OK, None, 1 << 30, 1 << 20, FAR, 2 * FAR, None) == 2
    assert q(BAD, None, 1, 32, FAR, 2 * FAR, None) == 3 and q(None, BAD, 1, 32, FAR, 2 * FAR, None) == 3
    assert q(OK, None, 1, 32, BAD, 2 * FAR, None) == 3
    assert q(OK, None, 1, 64, OK + 240, FAR, None) == 2 and q(OK, None, 1, 64, FAR, OK + 255, None) == 2
    assert q(OK, None, 1, 64, FAR, FAR + 31, None) == 2
    assert q(OK, None, 0, 32, FAR, 2 * FAR, None) == 0 and q(OK, None, 5, 0, FAR, 2 * FAR, None) == 0
    assert d(None, OK, 1, 32, FAR, None, None) == 1 and d(OK, None, 1, 32, FAR, None, None) == 1
    assert d(OK, OK, 1, 32, None, None, None) == 1 and d(OK, OK, 1, 32, FAR, 2 * FAR, None) == 1
    assert d(OK, OK, 1, 31, FAR, None, None) == 2 and d(OK, OK, 1, 32, BAD, None, None) == 3
    assert d(OK, 2 * FAR, 1, 32, OK, None, None) == 2 and d(2 * FAR, OK, 1, 32, OK, None, None) == 2
    assert d(OK, 2 * FAR, 0, 32, FAR, None, None) == 0


def test_the_quantiser_takes_no_more_than_a_grid_holds():
    # a thread for 32 values, less than 2^32 of them; a size that is taken ends at the misaligned address behind it
    q, d = lib.wq_quantize_mxfp4, lib.wq_dequantize_mxfp4
    for n, k, rc in [((1 << 32) - 256, 32, 3), ((1 << 32) - 255, 32, 2), (1 << 32, 32, 2), (1, (1 << 37) - (1 << 13), 3),
                     (1, 1 << 37, 2), (1 << 18, 1 << 20, 2), (1 << 20, 1 << 16, 3), (1 << 16, 1 << 22, 2)]:
        assert q(BAD, None, n, k, FAR, 2 * FAR, None) == rc and q(None, BAD, n, k, FAR, 2 * FAR, None) == rc
        assert d(OK, OK, n, k, BAD, None, None) == rc and d(OK, OK, n, k, None, BAD, None) == rc


def test_null_descriptions_and_foreign_plans():
    assert lib.wq_block_norm_prepare(None, OK) == 1
    for name in ("wq_gemm_mxfp4", "wq_moe_ffn"):
        assert getattr(lib, name + "_prepare")(None, OK, 0, OK) == 1
    for _, _, plan in CALLS.values():
        run = getattr(lib, plan.__name__.replace("_plan", "_run"))
        assert run(None, None) == 1
        assert run(ctypes.byref(plan()), None) == 2


def test_workspace_sizes():
    d, p = gemm(x=OK, m=64, k=4096, x_stride=4096), wq.wq_gemm_mxfp4_plan()
    need = wq.wq_gemm_mxfp4_workspace_bytes(64, 32, 4096)
    assert need > 16 == wq.wq_gemm_mxfp4_workspace_bytes(1, 32, 64)
    assert lib.wq_gemm_mxfp4_prepare(ctypes.byref(d), OK, need - 1, ctypes.byref(p)) == 2
    assert lib.wq_gemm_mxfp4_prepare(ctypes.byref(d), BAD, need, ctypes.byref(p)) == 3
    assert lib.wq_gemm_mxfp4_prepare(ctypes.byref(d), None, need, ctypes.byref(p)) == 1
    assert wq.wq_gemm_mxfp4_workspace_bytes(1, 32, 48) == 0 == wq.wq_gemm_mxfp4_workspace_bytes(-1, 32, 64)
    d, p = moe(x=OK), wq.wq_moe_ffn_plan()
    need = wq.wq_moe_ffn_workspace_bytes(3, 64, 32, 8, 2)
    assert need > 0
    assert lib.wq_moe_ffn_prepare(ctypes.byref(d), OK, need - 1, ctypes.byref(p)) == 2
    assert lib.wq_moe_ffn_prepare(ctypes.byref(d), BAD, need, ctypes.byref(p)) == 3
    assert wq.wq_moe_ffn_workspace_bytes(65, 64, 32, 8, 2) == 0 == wq.wq_moe_ffn_workspace_bytes(1, 64, 32, 2, 3)


def test_a_decode_step_does_not_take_mxfp4():
    plan = wq.wq_step_plan()
    mats = (wq.wq_matrix * 1)(wq.wq_matrix(OK, OK, OK, 32, 64, OK, None))
    assert lib.wq_decode_step_prepare(wq.WQ_FORMAT["mxfp4"], 1, mats, 1, OK, 1 << 20, ctypes.byref(plan)) == 2


def test_the_binding_refuses_host_tensors_types_and_shapes():
    x, b = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 32, dtype=torch.uint8)
    for call in (lambda: wq.wq_gemm_mxfp4_prepare(x, b, b, x), lambda: wq.wq_moe_ffn_prepare(x, b, b, b, b, x),
                 lambda: wq.wq_block_norm_prepare(x), lambda: wq.wq_quantize_mxfp4(None, x, 2, 64, b, b),
                 lambda: wq.wq_dequantize_mxfp4(b, b, 2, 64, None, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="uint8"):
        wq.wq_gemm_mxfp4_prepare(x, x, b, x)
    with pytest.raises(ValueError, match="float32"):
        wq.wq_block_norm_prepare(x.half())
    with pytest.raises(ValueError, match="axes"):
        wq.wq_block_norm_prepare(x[0])
    with pytest.raises(ValueError, match="bytes"):
        wq.wq_quantize_mxfp4(None, x, 2, 128, b, b)
    with pytest.raises(ValueError, match="tensor"):
        wq.wq_gemm_mxfp4_prepare(x, None, b, x)
