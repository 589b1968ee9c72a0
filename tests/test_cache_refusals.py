"""Refusals of the cache operators: host-visible mistakes give a status and need no device."""
import array
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_rejection_gb300 as sv

P = 0x10000  # an aligned address; nothing is read from it

STEP = dict(k_cache=P, v_cache=2 * P, k_page_stride=16 * 2 * 64, k_slot_stride=2 * 64, k_cache_head_stride=64,
            v_page_stride=16 * 2 * 64, v_slot_stride=2 * 64, v_cache_head_stride=64, page_table=P, table_stride=8, lengths=P,
            cu_num_draft=P, num_rows=9, num_reqs=3, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=20, page_size=16,
            pages_per_req=8, dtype=sv.SV_BF16, cache_dtype=sv.SV_BF16, device=1000)  # (no device has this ordinal)


def append_args(**kw):
    base = dict(STEP, q=P, k=P, v=P, q_out=3 * P, q_row_stride=256, q_head_stride=64, k_row_stride=128, k_head_stride=64,
                v_row_stride=128, v_head_stride=64, q_out_row_stride=256, q_out_head_stride=64, inv_freq=P, rotary_dim=64)
    return sv.CacheAppendArgs(**{**base, **kw})


def attention_args(**kw):
    base = dict(STEP, q=P, out=3 * P, lse=P, q_row_stride=256, q_head_stride=64, out_row_stride=256, out_head_stride=64,
                workspace=P, workspace_bytes=1 << 40, scale=0.125)
    return sv.CacheAttentionArgs(**{**base, **kw})


STEPS = [
    ({}, sv.SV_EDEVICE), (dict(device=-1), sv.SV_EDEVICE), (dict(cu_num_draft=None), sv.SV_EDEVICE),
    (dict(num_rows=0, k_cache=None, lengths=None), sv.SV_OK), (dict(num_reqs=0, page_table=None), sv.SV_OK),
    (dict(num_rows=-1), sv.SV_EINVAL), (dict(num_reqs=-1), sv.SV_EINVAL), (dict(num_pages=-1), sv.SV_EINVAL),
    (dict(page_size=0), sv.SV_EINVAL), (dict(page_size=sv.SV_MAX_PAGE + 1), sv.SV_ECAPACITY), (dict(pages_per_req=-1), sv.SV_EINVAL),
    (dict(pages_per_req=9), sv.SV_EINVAL), (dict(table_stride=1 << 41), sv.SV_EINVAL), (dict(num_kv_heads=0), sv.SV_EINVAL),
    (dict(dtype=sv.SV_F32), sv.SV_EDTYPE), (dict(dtype=sv.SV_E4M3), sv.SV_EDTYPE), (dict(cache_dtype=sv.SV_F16), sv.SV_EDTYPE),
    (dict(cache_dtype=sv.SV_F32), sv.SV_EDTYPE), (dict(dtype=sv.SV_F16), sv.SV_EDTYPE),
    (dict(dtype=sv.SV_F16, cache_dtype=sv.SV_F16), sv.SV_EDEVICE), (dict(cache_dtype=sv.SV_E4M3), sv.SV_EDEVICE),
    (dict(k_scale=P), sv.SV_EINVAL), (dict(cache_dtype=sv.SV_E4M3, k_scale=P, v_scale=P), sv.SV_EDEVICE),
    (dict(cache_dtype=sv.SV_E4M3, v_scale=P + 2), sv.SV_EINVAL), (dict(k_cache=None), sv.SV_EINVAL), (dict(v_cache=None), sv.SV_EINVAL),
    (dict(k_cache=P + 8), sv.SV_EINVAL), (dict(k_slot_stride=132), sv.SV_EINVAL), (dict(v_cache_head_stride=-64), sv.SV_EINVAL),
    (dict(k_page_stride=1 << 60), sv.SV_EINVAL), (dict(cache_dtype=sv.SV_E4M3, k_slot_stride=136), sv.SV_EINVAL),
    (dict(page_table=None), sv.SV_EINVAL), (dict(lengths=None), sv.SV_EINVAL), (dict(lengths=P + 1), sv.SV_EINVAL),
    (dict(cu_num_draft=P + 2), sv.SV_EINVAL), (dict(page_table=P + 2), sv.SV_EINVAL), (dict(q=P + 8), sv.SV_EINVAL),
    (dict(q=None), sv.SV_EINVAL), (dict(q_row_stride=252), sv.SV_EINVAL), (dict(q_head_stride=-64), sv.SV_EINVAL),
    (dict(num_pages=0, k_cache=None, v_cache=None), sv.SV_EDEVICE),
]


@pytest.mark.parametrize("change,status", STEPS + [
    (dict(head_dim=24), sv.SV_EINVAL), (dict(head_dim=0), sv.SV_EINVAL), (dict(head_dim=272, rotary_dim=64), sv.SV_ECAPACITY),
    (dict(rotary_dim=24), sv.SV_EINVAL), (dict(rotary_dim=80), sv.SV_EINVAL), (dict(rotary_dim=-16), sv.SV_EINVAL),
    (dict(inv_freq=None), sv.SV_EINVAL), (dict(inv_freq=None, rotary_dim=0), sv.SV_EDEVICE), (dict(inv_freq=P + 2), sv.SV_EINVAL),
    (dict(positions=P), sv.SV_EINVAL), (dict(positions=P, num_axes=1), sv.SV_EDEVICE),
    (dict(positions=P, num_axes=3, positions_stride=8), sv.SV_EINVAL), (dict(positions=P, num_axes=3, positions_stride=9), sv.SV_EDEVICE),
    (dict(positions=P, num_axes=5, positions_stride=9), sv.SV_ECAPACITY), (dict(axes=bytes(32)), sv.SV_EINVAL),
    (dict(axes=bytes([0] * 31 + [2]), positions=P, num_axes=2, positions_stride=9), sv.SV_EINVAL),
    (dict(axes=bytes([0] * 31 + [1]), positions=P, num_axes=2, positions_stride=9), sv.SV_EDEVICE),
    (dict(k=None), sv.SV_EINVAL), (dict(v=None), sv.SV_EINVAL), (dict(v=P + 4), sv.SV_EINVAL), (dict(q_out=None), sv.SV_EINVAL),
    (dict(num_q_heads=0, q=None, q_out=None), sv.SV_EDEVICE), (dict(num_q_heads=0, q=None, q_out=None, q_row_stride=0, q_out_row_stride=0), sv.SV_EDEVICE), (dict(num_q_heads=-1), sv.SV_EINVAL),
    (dict(q_out=P), sv.SV_EDEVICE), (dict(q_out=P, q_out_row_stride=264), sv.SV_EINVAL), (dict(q_out_row_stride=128), sv.SV_EINVAL),
    (dict(k_cache_head_stride=0), sv.SV_EINVAL), (dict(v_slot_stride=64), sv.SV_EINVAL), (dict(k_row_stride=0), sv.SV_EDEVICE),
    (dict(v_cache=P), sv.SV_EINVAL),
])
def test_append_refuses(change, status):
    assert sv.lib().spec_verify_cache_append(ctypes.byref(append_args(**change)), None) == status


@pytest.mark.parametrize("change,status", STEPS + [
    (dict(head_dim=80), sv.SV_EINVAL), (dict(head_dim=512), sv.SV_EINVAL), (dict(num_q_heads=5), sv.SV_EINVAL),
    (dict(num_q_heads=0), sv.SV_EINVAL), (dict(window=-1), sv.SV_EINVAL), (dict(scale=float("nan")), sv.SV_EINVAL),
    (dict(scale=float("inf")), sv.SV_EINVAL), (dict(out=None), sv.SV_EINVAL), (dict(out=P), sv.SV_EINVAL), (dict(out=P + 4), sv.SV_EINVAL),
    (dict(num_q_heads=1 << 20, num_kv_heads=1, num_rows=1 << 12, num_reqs=1), sv.SV_ECAPACITY), (dict(pages_per_req=1 << 20, page_size=1 << 11, table_stride=1 << 20), sv.SV_ECAPACITY),
    (dict(lse=P + 2), sv.SV_EINVAL), (dict(lse=None), sv.SV_EDEVICE), (dict(workspace=P + 8), sv.SV_EINVAL),
    (dict(out_head_stride=32), sv.SV_EINVAL), (dict(out_row_stride=0), sv.SV_EINVAL), (dict(k_page_stride=0), sv.SV_EINVAL), (dict(q_row_stride=0), sv.SV_EINVAL),
])
def test_attention_refuses(change, status):
    assert sv.lib().spec_verify_cache_attention(ctypes.byref(attention_args(**change)), None) == status


def test_null_arguments():
    n = ctypes.c_int64()
    assert sv.lib().spec_verify_cache_append(None, None) == sv.SV_EINVAL
    assert sv.lib().spec_verify_cache_attention(None, None) == sv.SV_EINVAL
    assert sv.lib().spec_verify_cache_attention_workspace(None, ctypes.byref(n)) == sv.SV_EINVAL
    assert sv.lib().spec_verify_cache_attention_workspace(ctypes.byref(attention_args()), None) == sv.SV_EINVAL


def test_workspace_goes_by_sizes_alone():
    args = attention_args(q=None, out=None, k_cache=None, v_cache=None, page_table=None, lengths=None, workspace=None, workspace_bytes=0, pages_per_req=100, table_stride=100)
    assert 0 < sv.spec_verify_cache_attention_workspace(args) <= sv.SV_CACHE_WORKSPACE
    one_tile = attention_args(pages_per_req=8, page_size=16)
    assert sv.spec_verify_cache_attention_workspace(one_tile) == 0   # (nothing to join)
    most = max(sv.spec_verify_cache_attention_workspace(attention_args(head_dim=d, num_q_heads=2 * g, num_rows=3000, num_reqs=300, page_size=64,
                                                                       pages_per_req=4000, table_stride=4000, cache_dtype=c))
               for d in (64, 128, 256) for g in (1, 2, 3, 5, 6, 7, 8, 16) for c in (sv.SV_BF16, sv.SV_E4M3))
    assert most == sv.SV_CACHE_WORKSPACE
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_verify_cache_attention_workspace(attention_args(head_dim=65))


# the binding: its checks come before any device is touched

def fake(shape, dtype=torch.bfloat16, device="cuda:0"):
    class On:  # a tensor of the CPU that says it is on the GPU
        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            told = {"device": torch.device(device), "is_cuda": device != "cpu", "get_device": lambda: torch.device(device).index if device != "cpu" else -1}
            return told[name] if name in told else getattr(self.t, name)

    return On(torch.zeros(shape, dtype=dtype))


def good():
    i32 = torch.int32
    return dict(k=fake((9, 2, 64)), v=fake((9, 2, 64)), q=fake((9, 4, 64)), k_cache=fake((20, 16, 2, 64)), v_cache=fake((20, 16, 2, 64)),
                page_table=fake((3, 8), i32), lengths=fake((3,), i32), cu_num_draft=fake((4,), i32), out=fake((9, 4, 64)), inv_freq=fake((32,), torch.float32))


BINDING = [
    dict(k_cache=fake((20, 16, 2, 128))), dict(v_cache=fake((20, 16, 3, 64))), dict(v_cache=fake((20, 16, 2, 64), torch.float16)),
    dict(k_cache=fake((20, 2, 64))), dict(page_table=fake((2, 8), torch.int32)), dict(page_table=fake((3, 8), torch.int64)),
    dict(lengths=fake((3,), torch.int64)), dict(lengths=fake((3, 1), torch.int32)), dict(cu_num_draft=fake((3,), torch.int32)),
    dict(q=fake((9, 4, 128))), dict(q=fake((9, 4))), dict(q=fake((9, 4, 64), torch.float16)), dict(out=fake((8, 4, 64))),
    dict(k_cache=fake((20, 16, 2, 64), device="cuda:1")), dict(page_table=fake((3, 8), torch.int32, "cpu")),
    dict(k_scale=fake((2,), torch.float32)), dict(q=fake((9, 4, 64), torch.float32)),
]


@pytest.mark.parametrize("change", BINDING + [
    dict(k=fake((9, 2, 64), device="cpu")), dict(k=fake((9, 2, 64), torch.float32)), dict(v=fake((9, 1, 64))), dict(inv_freq=fake((32,), torch.float64)),
    dict(positions=fake((3, 8), torch.int32)), dict(positions=fake((1, 9), torch.int64)), dict(axes=[0] * 31), dict(q=None), dict(axes=[0] * 31 + [300]),
])
def test_append_binding_refuses(change):
    a = {**good(), **change}
    with pytest.raises(ValueError):
        sv.cache_append(a.pop("k"), a.pop("v"), a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"), a.pop("lengths"), stream=0, **a)


@pytest.mark.parametrize("change", BINDING + [
    dict(q=fake((9, 3, 64))), dict(lse=True), dict(cu_num_draft=None, lengths=fake((30,), torch.int32), page_table=fake((30, 8), torch.int32)),
])
def test_attention_binding_refuses(change):
    a = {**good(), **change}
    for name in ("k", "v", "inv_freq"):
        a.pop(name)
    with pytest.raises(ValueError):
        sv.cache_attention(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"), a.pop("lengths"), out=[a.pop("out")], stream=0, **a)


def test_binding_refuses_what_32_bits_do_not_hold():
    many = dict(k_cache=fake((1, 16, 2, 64)), v_cache=fake((1, 16, 2, 64)))
    many = {name: type(t)(t.t.expand(2**32 + 1, -1, -1, -1)) for name, t in many.items()}
    table = fake((3, 1), torch.int32)
    for change in (many, dict(page_table=type(table)(table.t.expand(-1, 2**32 + 1)))):
        test_append_binding_refuses(change)
        test_attention_binding_refuses(change)
    for window in (2**31, 2**32 + 5, -1, 5 - 2**32):
        test_attention_binding_refuses(dict(window=window))


def axes_sent(axes, monkeypatch):
    """The axes that a call with these axes hands to the library (which is not called)."""
    got = []

    def call(ref, stream):
        args = ref._obj
        got.append(list(ctypes.string_at(ctypes.c_void_p.from_buffer(args, sv.CacheAppendArgs.axes.offset).value, args.rotary_dim // 2)))
        return sv.SV_OK

    monkeypatch.setattr(sv._cache_torch(), "append", call)
    a = dict(good(), positions=fake((3, 9), torch.int32), axes=axes)
    sv.cache_append(a.pop("k"), a.pop("v"), a.pop("k_cache"), a.pop("v_cache"), a.pop("page_table"), a.pop("lengths"), stream=0, **a)
    return got[0]


@pytest.mark.parametrize("kind", ("list", "tuple", "bytes", "array.array", "int8", "int32", "int64", "uint64", "strided", "tensor32", "tensor64"))
def test_axes_are_numbers_whatever_holds_them(kind, monkeypatch):
    want = [m % 3 for m in range(32)] if kind == "strided" else [0] * 8 + [1] * 12 + [2] * 12
    held = {"list": list, "tuple": tuple, "bytes": bytes, "array.array": lambda a: array.array("l", a),
            "strided": lambda a: np.array(a + a, dtype=np.int32).reshape(2, 32).T.copy()[:, 0],
            "tensor32": lambda a: torch.tensor(a, dtype=torch.int32), "tensor64": torch.tensor}
    make = held.get(kind) or (lambda a: np.array(a, dtype=kind))
    assert axes_sent(make(want), monkeypatch) == want


@pytest.mark.parametrize("axes", (np.full(32, 0.5), np.zeros((32, 2), dtype=np.int64), torch.zeros(32), ["0"] * 32, "0" * 32, np.full(32, -1), np.full(32, 256)))
def test_axes_that_are_no_axis_numbers_are_refused(axes, monkeypatch):
    with pytest.raises(ValueError):
        axes_sent(axes, monkeypatch)


def test_error_word_of_the_cache_operators():
    assert sv.lib().spec_verify_cache_last_error(None) == sv.SV_EINVAL
    with open(sv._HEADER, encoding="utf-8") as f:
        assert f"#define SV_ERR_WAIT {sv.SV_ERR_WAIT}u" in f.read()
    if not torch.cuda.is_available():
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.spec_verify_cache_last_error()
        assert e.value.status == sv.SV_EDEVICE
