"""Refusals of the verify-pass calls that need no GPU: C argument checks (fake,
misaligned addresses that no call may reach) and the binding's tensor checks."""

import ctypes

import pytest
import torch

import weight_only_quantized_wq_amd as wq

from oracle import verify
from weight_only_quantized_wq_amd import _binding

BAD = 0x1001
OK = 0x2000
lib = _binding.lib


def cache(**kw):
    f = dict(k=OK, v=OK, pages=4, page_size=16, page_stride=2048, token_stride=128, head_stride=64, table=OK,
             table_width=4, table_stride=4, kv_heads=2, head_dim=64)
    f.update(kw)
    return wq.wq_kv_cache(*(f[n] for n, _ in wq.wq_kv_cache._fields_))


def batch(**kw):
    f = dict(starts=OK, lengths=OK, tokens=5, requests=2)
    f.update(kw)
    return wq.wq_batch(*(f[n] for n, _ in wq.wq_batch._fields_))


def _fill(cls, defaults, kw):
    defaults.update(kw)
    assert set(defaults) == {n for n, _ in cls._fields_}
    return cls(**defaults)


def rope(**kw):
    return _fill(wq.wq_qkv_rope, dict(cache=cache(), batch=batch(), qkv_f32=None, qkv_bf16=OK, qkv_stride=512, q=BAD,
                                      q_stride=256, positions=OK, q_norm=OK, k_norm=OK, freq=OK, eps=1e-6,
                                      rot_scale=1.0, rot_dim=64, interleaved=0, heads=4), kw)


def attention(**kw):
    return _fill(wq.wq_tree_attention, dict(cache=cache(), batch=batch(), q=OK, q_stride=256, y=BAD, y_stride=256,
                                            tree=OK, scale=0.125, heads=4, max_tokens=5), kw)


def accept(**kw):
    return _fill(wq.wq_kv_accept, dict(cache=cache(k=BAD), layers=2, layer_stride=8192, requests=2, lengths=OK, path=OK,
                                       path_width=5, path_stride=5, accepted=OK), kw)


def lora(**kw):
    return _fill(wq.wq_lora, dict(x=BAD, x_stride=64, base=OK, base_stride=32, y_f32=OK, y_bf16=None, y_stride=32, a=OK,
                                  b=OK, adapter=OK, ranks=OK, scale=OK, tokens=3, k=64, n=32, adapters=2, rank=8), kw)


CALLS = {
    "rope": (rope, lambda d, p: lib.wq_qkv_rope_prepare(ctypes.byref(d), ctypes.byref(p)), wq.wq_qkv_rope_plan),
    "attention": (attention, lambda d, p: lib.wq_tree_attention_prepare(ctypes.byref(d), OK, 1 << 40, ctypes.byref(p)),
                  wq.wq_tree_attention_plan),
    "accept": (accept, lambda d, p: lib.wq_kv_accept_prepare(ctypes.byref(d), ctypes.byref(p)), wq.wq_kv_accept_plan),
    "lora": (lora, lambda d, p: lib.wq_lora_prepare(ctypes.byref(d), OK, 1 << 40, ctypes.byref(p)), wq.wq_lora_plan),
}


def status(call, **kw):
    make, prepare, plan = CALLS[call]
    return prepare(make(**kw), plan())


@pytest.mark.parametrize("call", CALLS)
def test_a_good_description_stops_only_at_its_misaligned_pointer(call):
    # every size is right, so the check that follows the sizes is the one that refuses
    assert status(call) == 3
    assert "aligned" in wq.last_error()


CACHE_SIZES = [dict(pages=0), dict(page_size=0), dict(page_size=-1), dict(table_width=0), dict(table_stride=3),
               dict(page_size=1 << 20, table_width=1 << 11, table_stride=1 << 11), dict(kv_heads=0),
               dict(kv_heads=1025), dict(head_dim=60), dict(head_dim=264), dict(head_dim=0), dict(page_stride=4),
               dict(token_stride=-8), dict(head_stride=12)]


@pytest.mark.parametrize("call", ["rope", "attention", "accept"])
@pytest.mark.parametrize("kw", CACHE_SIZES, ids=str)
def test_cache_sizes(call, kw):
    assert status(call, cache=cache(**kw)) == 2


@pytest.mark.parametrize("call", ["rope", "attention", "accept"])
@pytest.mark.parametrize("name", ["k", "v", "table"])
def test_cache_null(call, name):
    assert status(call, cache=cache(**{name: None})) == 1


@pytest.mark.parametrize("call", ["rope", "attention"])
@pytest.mark.parametrize("kw,rc", [(dict(starts=None), 1), (dict(lengths=None), 1), (dict(tokens=-1), 2),
                                   (dict(tokens=(1 << 20) + 1), 2), (dict(requests=-1), 2), (dict(requests=4097), 2)],
                         ids=str)
def test_batch(call, kw, rc):
    assert status(call, batch=batch(**kw)) == rc


@pytest.mark.parametrize("call,kw,rc", [
    ("rope", dict(q=None), 1), ("rope", dict(qkv_bf16=None), 1), ("rope", dict(qkv_f32=OK), 1),
    ("rope", dict(freq=None), 1), ("rope", dict(heads=3), 2), ("rope", dict(heads=0), 2), ("rope", dict(heads=2048), 2),
    ("rope", dict(rot_dim=-2), 2), ("rope", dict(rot_dim=7), 2), ("rope", dict(rot_dim=66), 2),
    ("rope", dict(qkv_stride=504), 2), ("rope", dict(qkv_stride=516), 2), ("rope", dict(q_stride=248), 2),
    ("rope", dict(q_stride=260), 2), ("rope", dict(eps=-1.0), 2), ("rope", dict(eps=float("nan")), 2),
    ("rope", dict(rot_scale=float("inf")), 2), ("rope", dict(q=OK, q_norm=BAD), 3),
    ("rope", dict(qkv_bf16=None, qkv_f32=OK, qkv_stride=514), 2),
    ("attention", dict(batch=batch(requests=4096), cache=cache(kv_heads=1024, head_stride=64, table_width=1 << 16,
                                                              table_stride=1 << 16), heads=1024, q_stride=65536,
                       y_stride=65536), 2),
    ("attention", dict(q=None), 1), ("attention", dict(y=None), 1), ("attention", dict(heads=5), 2),
    ("attention", dict(heads=0), 2), ("attention", dict(heads=130), 2), ("attention", dict(max_tokens=0), 2),
    ("attention", dict(max_tokens=65), 2), ("attention", dict(cache=cache(head_dim=72)), 2),
    ("attention", dict(q_stride=248), 2), ("attention", dict(y_stride=252), 2),
    ("attention", dict(scale=float("nan")), 2), ("attention", dict(y=OK), 2), ("attention", dict(y=0x3000, tree=BAD), 3),
    ("accept", dict(lengths=None), 1), ("accept", dict(path=None), 1), ("accept", dict(accepted=None), 1),
    ("accept", dict(layers=0), 2), ("accept", dict(layers=4097), 2), ("accept", dict(layer_stride=4), 2),
    ("accept", dict(requests=4097), 2), ("accept", dict(path_width=0), 2), ("accept", dict(path_width=65, path_stride=65), 2),
    ("accept", dict(path_stride=4), 2),
    ("lora", dict(x=None), 1), ("lora", dict(a=None), 1), ("lora", dict(b=None), 1), ("lora", dict(adapter=None), 1),
    ("lora", dict(y_f32=None), 1), ("lora", dict(k=60), 2), ("lora", dict(k=0), 2), ("lora", dict(k=65544, x_stride=65544), 2),
    ("lora", dict(rank=12), 2), ("lora", dict(rank=136), 2), ("lora", dict(rank=0), 2), ("lora", dict(adapters=0), 2),
    ("lora", dict(adapters=4097), 2), ("lora", dict(tokens=4097), 2), ("lora", dict(tokens=-1), 2), ("lora", dict(n=-1), 2),
    ("lora", dict(x_stride=56), 2), ("lora", dict(x_stride=68), 2), ("lora", dict(y_stride=31), 2),
    ("lora", dict(base_stride=31), 2), ("lora", dict(y_stride=40), 2), ("lora", dict(x=OK, base=BAD), 3),
], ids=str)
def test_refusals(call, kw, rc):
    assert status(call, **kw) == rc, wq.last_error()


def test_null_descriptions_and_foreign_plans():
    for name in ("wq_qkv_rope", "wq_kv_accept"):
        assert getattr(lib, name + "_prepare")(None, OK) == 1
    for name in ("wq_tree_attention", "wq_lora"):
        assert getattr(lib, name + "_prepare")(None, OK, 0, OK) == 1
    for call, (_, _, plan) in CALLS.items():
        run = getattr(lib, plan.__name__.replace("_plan", "_run"))
        assert run(None, None) == 1
        assert run(ctypes.byref(plan()), None) == 2


def test_workspace_sizes():
    d, p = attention(y=0x3000), wq.wq_tree_attention_plan()
    need = wq.wq_tree_attention_workspace_bytes(2, 4, 2, 64, 5)
    assert need > 0
    assert lib.wq_tree_attention_prepare(ctypes.byref(d), OK, need - 1, ctypes.byref(p)) == 2
    assert lib.wq_tree_attention_prepare(ctypes.byref(d), BAD, need, ctypes.byref(p)) == 3
    assert lib.wq_tree_attention_prepare(ctypes.byref(d), None, need, ctypes.byref(p)) == 1
    assert wq.wq_tree_attention_workspace_bytes(2, 5, 2, 64, 5) == 0
    assert wq.wq_tree_attention_workspace_bytes(2, 4, 2, 80, 5) == 0
    d, p = lora(x=OK), wq.wq_lora_plan()
    need = wq.wq_lora_workspace_bytes(3, 64, 2, 8)
    assert need > 0
    assert lib.wq_lora_prepare(ctypes.byref(d), OK, need - 1, ctypes.byref(p)) == 2
    assert lib.wq_lora_prepare(ctypes.byref(d), BAD, need, ctypes.byref(p)) == 3
    assert wq.wq_lora_workspace_bytes(3, 60, 2, 8) == 0


@pytest.mark.parametrize("args", [(9, 64, 1e4), (0, 7, 1e4), (0, 0, 1e4), (0, 258, 1e4), (0, 64, 1.0), (1, 64, 1e4, 0.5),
                                  (2, 64, 1e4, 8.0, 4.0, 4.0), (2, 64, 1e4, 8.0, 0.0, 4.0),
                                  (3, 64, 1e4, 8.0, 1.0, 32.0, 0.5), (1, 64, 1e4, float("nan"))], ids=str)
def test_rope_frequency_refusals(args):
    kind, rot_dim, base = args[:3]
    with pytest.raises(wq.WQError):
        wq.wq_rope_frequencies(rot_dim, base, kind, *args[3:])


def test_the_binding_refuses_host_tensors_types_and_shapes():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        wq.wq_lora_prepare(x, x, x, x, x)
    with pytest.raises(ValueError, match="float32"):
        wq.wq_qkv_rope_prepare(x.half(), x, x, x, x, x, x)
    with pytest.raises(ValueError, match="axes"):
        wq.wq_qkv_rope_prepare(x[0], x, x, x, x, x, x)
    with pytest.raises(ValueError, match="contiguous"):
        wq.wq_lora_prepare(x[:, ::2], x, x, x, x)
    with pytest.raises(ValueError, match="tensor"):
        wq.wq_kv_accept_prepare(None, None, None, None, None, None)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_many_requests_take_a_kernel_whose_buffers_leave_room(dim):
    # beside the largest blocks' buffers there is LDS for the sums of 2048 requests: more take blocks of 64 rows
    assert wq.wq_tree_attention_workspace_bytes(2049, 32, 4, dim, 64) == wq.wq_tree_attention_workspace_bytes(
        2049, 4, 4, dim, 64) == wq.wq_tree_attention_workspace_bytes(4096, 32, 4, dim, 64)


@pytest.mark.parametrize("width,rc", [(507 * 32, 3), (507 * 32 + 1, 2), (509 * 32, 2)])
def test_the_deal_of_the_largest_batches_stays_in_32_bits(width, rc):
    # 4096 requests x 1024 key heads x (tiles + 4) < 2^31, so fewer than 508 tiles of 32 positions; y is misaligned
    assert status("attention", batch=batch(requests=4096), heads=1024, q_stride=65536, y_stride=65536, max_tokens=1,
                  cache=cache(kv_heads=1024, head_stride=64, page_size=1, table_width=width, table_stride=width)) == rc


@pytest.mark.parametrize("layers,rc", [(1, 3), (2, 2)])
def test_layers_must_not_lie_on_each_other(layers, rc):
    # a row that one layer's copy overwrites could be another's source; the k of a lone layer is only misaligned
    assert status("accept", layers=layers, layer_stride=0) == rc


# rows of 4 heads of 64 (512 bytes) beside rows of 8 (q | k | v, 1024 bytes), five of them
MEET = [
    ("rope", dict(q=OK, qkv_bf16=OK)),                                                     # in place
    ("rope", dict(q=OK + 4096, qkv_bf16=OK)),                                              # the last row
    ("rope", dict(q=OK, qkv_bf16=OK + 4 * 512)),                                           # the first
    ("rope", dict(q=OK, qkv_bf16=None, qkv_f32=OK + 4 * 512, qkv_stride=512)),
    ("rope", dict(q=OK + 1008, qkv_bf16=OK, q_stride=768, qkv_stride=768)),                # columns of one buffer, 8 of them shared
    ("rope", dict(q=OK + 5 * 1536 - 16, qkv_bf16=OK + 1008, q_stride=256, qkv_stride=768)),
    ("rope", dict(q=OK + 1024, qkv_bf16=OK, q_stride=776, qkv_stride=768)),                # strides that drift apart, row 33
    ("attention", dict(q=OK, y=OK + 4 * 512)),
    ("attention", dict(q=OK + 16, y=OK)),
    ("attention", dict(q=OK + 496, y=OK, q_stride=512, y_stride=512)),
    ("lora", dict(x=OK, y_f32=OK + 256)),                                                  # x: 3 rows of 128 bytes
    ("lora", dict(x=OK, y_f32=None, base=None, y_bf16=OK, y_stride=64)),                   # y in place of x
    ("lora", dict(x=OK, y_f32=OK + 0x1000 - 16, a=OK + 0x1000)),
    ("lora", dict(x=OK, y_f32=OK + 0x2000, b=OK + 0x2000)),
    ("lora", dict(x=OK, y_f32=OK + 0x3000, adapter=OK + 0x3000 + 380)),
    ("lora", dict(x=OK, y_f32=OK + 0x3000, ranks=OK + 0x3000)),
    ("lora", dict(x=OK, y_f32=OK + 0x3000, scale=OK + 0x3000)),
    ("lora", dict(x=OK, y_f32=OK + 0x3000, y_bf16=OK + 0x3000 + 376)),
    ("lora", dict(x=OK, y_f32=OK + 0x3000, base=OK + 0x3000 + 128)),                       # base a row on
    ("lora", dict(x=OK, y_f32=None, y_bf16=OK + 0x3000, base=OK + 0x3000)),
]
APART = [
    ("rope", dict(q=OK + 5 * 1024, qkv_bf16=OK)), ("rope", dict(q=OK, qkv_bf16=OK + 5 * 512)),
    ("rope", dict(q=OK + 1024, qkv_bf16=OK, q_stride=768, qkv_stride=768)),                # columns of one buffer
    ("rope", dict(q=OK, qkv_bf16=OK + 512, q_stride=768, qkv_stride=768)),
    ("rope", dict(q=OK + 1024, qkv_bf16=OK, q_stride=768, qkv_stride=768, batch=batch(tokens=1 << 20))),
    ("attention", dict(q=OK, y=OK + 5 * 512)), ("attention", dict(q=OK + 512, y=OK, q_stride=512, y_stride=512)),
    ("attention", dict(q=OK, y=OK, batch=batch(tokens=0))),
    ("lora", dict(x=OK, base=0x13000, y_f32=0x13000, a=0x20000, b=0x30000)),               # base in place
    ("lora", dict(x=OK, base=0x13080, y_f32=0x13000, a=0x20000, b=0x30000, y_stride=64, base_stride=64)),
    ("lora", dict(x=OK, base=0x13000, y_f32=0x13000, y_bf16=0x13180, a=0x20000, b=0x30000)),
]


def room(call, kw):
    """Inputs of their own for adapters, unless the case says otherwise."""
    return dict(dict(base=0x40000, a=0x20000, b=0x30000, adapter=0x50000, ranks=0x51000, scale=0x52000), **kw) if call == "lora" else kw


@pytest.mark.parametrize("call,kw", MEET, ids=str)
def test_results_must_not_lie_on_what_is_read(call, kw):
    if kw.get("q_stride") == 776:
        kw = dict(kw, batch=batch(tokens=34))
    assert status(call, **room(call, kw)) == 2
    assert "overlap" in wq.last_error() or "y must not be q" in wq.last_error()


@pytest.mark.parametrize("call,kw", APART, ids=str)
def test_results_beside_what_is_read(call, kw):
    # accepted, or refused only for want of a device
    assert status(call, **room(call, kw)) in (0, 4), wq.last_error()


@pytest.mark.parametrize("kind,high", [("bands", 4.0), (2, 4.0), ("ramp", 32.0), (3, 32.0)])
def test_rope_frequency_turns_that_a_kind_is_published_with(kind, high):
    got, scale = wq.wq_rope_frequencies(128, 10000.0, kind, factor=8.0, original=4096.0)
    want, want_scale = verify.rope_frequencies({2: "bands", 3: "ramp"}.get(kind, kind), 128, 10000.0, 8.0, 1.0, high, 4096.0)
    assert torch.all((got.double() - torch.from_numpy(want)).abs() <= 2.0 ** -23 * torch.from_numpy(want))
    assert abs(scale - want_scale) <= 2.0 ** -24 * want_scale


@pytest.mark.parametrize("name", ["adapter", "ranks", "scale", "a", "b"])
@pytest.mark.timeout(20, method="thread")
def test_inputs_between_the_rows_of_a_padded_result(name):
    # results of 128 bytes every 512 (b: every 2048): an input of one piece in the gap behind the first or second row
    wide = 512 if name in ("a", "b") else 128
    for row in (0, 1):
        kw = dict(x=OK, y_f32=0x13000, y_stride=wide, k=8, x_stride=8, **{name: 0x13000 + row * 4 * wide + 144})
        assert status("lora", **room("lora", kw)) in (0, 4), wq.last_error()
        kw[name] = 0x13000 + row * 4 * wide + 112
        assert status("lora", **room("lora", kw)) == (3 if name in ("a", "b") and kw[name] % 16 else 2)
