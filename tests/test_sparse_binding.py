"""What the Python binding of the sparse decode step's calls checks, on the CPU:
the extension is pointed at entry points that only note their arguments, and at
tensors that claim a device."""
import ctypes as C

import pytest
import torch

import bit_paged_kv_gb300 as saw
from bit_paged_kv_gb300 import build as saw_build
from test_binding_checks import HERE, On, cache, i32, rows

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("saw_norm_rope_append", "saw_page_summary", "saw_select_pages", "saw_sparse_decode_int4")


@pytest.fixture(scope="module")
def calls():
    saw_build.build()
    L, seen = saw.lib(), []
    m = saw._binding._bind_step()
    fakes = [C.CFUNCTYPE(C.c_int32, *getattr(L, n).argtypes)(lambda *a, n=n: seen.append((n, a)) or 0) for n in NAMES]
    plain = [getattr(L, n) for n in ("saw_build_tables", "saw_rope_table", "saw_rope_append", "saw_prefix_decode_int4",
                                     "saw_cache_bytes")]
    at = lambda fs: [C.cast(f, C.c_void_p).value for f in fs]
    m.init(*at(plain), torch.int32, F32, BF, F16, lambda: HERE, lambda dev: 77)
    m.init_sparse(*at([*fakes, L.saw_summary_bytes]))
    yield seen
    saw._binding._bind_step()  # the library's entry points again


def summary(pages=4, hkv=2, d=128):
    return On(torch.zeros(saw.saw_summary_bytes(pages, hkv, d), dtype=torch.uint8))


def norm_args():
    return dict(q=rows(3, 4, 128), k=rows(3, 2, 128), v=rows(3, 2, 128), q_weight=rows(128), k_weight=rows(128),
                positions=i32(3), cos_sin=On(torch.zeros(8, 128)), slot_mapping=i32(3), q_out=rows(3, 4, 128),
                k_cache=cache(), v_cache=cache(), num_pages=4, page_size=16, rotate_k=True, rotate_v=True, block_h=128,
                eps=1e-5, weight_offset=1.0, dev_status=i32(1))


def summary_args():
    return dict(k_cache=cache(), block_tables=i32(3, 4), seq_lens=i32(3), new_lens=i32(3), max_new_len=16,
                num_kv_heads=2, head_dim=128, num_pages=4, page_size=16, summary=summary(), dev_status=i32(1))


def select_args():
    return dict(q=rows(3, 4, 128), summary=summary(), block_tables=i32(3, 4), seq_lens=i32(3), max_seq_len=64,
                num_kv_heads=2, num_pages=4, page_size=16, rotate_k=True, block_h=128, first_pages=1, last_pages=1,
                sel_tables=i32(3, 2, 3), sel_lens=i32(3, 2), sel_pages=i32(3, 2, 3), dev_status=i32(1))


def sparse_args():
    return dict(q=rows(3, 4, 128), k_cache=cache(), v_cache=cache(), sel_tables=i32(3, 2, 4), sel_lens=i32(3, 2),
                max_sel_len=64, num_kv_heads=2, num_pages=4, page_size=16, rotate_k=True, rotate_v=True, block_h=128,
                out=rows(3, 4, 128), workspace=On(torch.zeros(64, dtype=torch.uint8)), dev_status=i32(1))


CALLS = {"norm": (saw.saw_norm_rope_append, norm_args), "summary": (saw.saw_page_summary, summary_args),
         "select": (saw.saw_select_pages, select_args), "sparse": (saw.saw_sparse_decode_int4, sparse_args)}
TENSORS = [(c, k) for c, (_, args) in CALLS.items() for k, v in args().items() if isinstance(v, On)]
OPTIONAL = [("norm", "q_weight"), ("norm", "k_weight"), ("norm", "dev_status"), ("summary", "new_lens"),
            ("summary", "dev_status"), ("select", "sel_pages"), ("select", "dev_status"), ("sparse", "workspace"),
            ("sparse", "dev_status")]


def refused(calls, name, args, text, error=ValueError):
    n = len(calls)
    with pytest.raises(error, match=text):
        CALLS[name][0](**args)
    assert len(calls) == n


@pytest.mark.parametrize("name", CALLS)
def test_the_arguments_pass(calls, name):
    n, args = len(calls), CALLS[name][1]()
    CALLS[name][0](**args)
    assert len(calls) == n + 1
    passed = calls[-1][1]
    assert passed[-1] == 77  # the stream
    for v in args.values():
        if isinstance(v, On):
            assert v.t.data_ptr() in passed


@pytest.mark.parametrize("dev", [-1, HERE + 1])
@pytest.mark.parametrize("name,arg", TENSORS)
def test_a_tensor_elsewhere_is_refused(calls, name, arg, dev):
    args = CALLS[name][1]()
    args[arg] = On(args[arg].t, dev)
    refused(calls, name, args, f"{arg} must be on cuda:{HERE}|current device is cuda:{HERE}|on a CUDA device")


@pytest.mark.parametrize("name,arg", OPTIONAL)
def test_what_may_be_left_out(calls, name, arg):
    n = len(calls)
    CALLS[name][0](**dict(CALLS[name][1](), **{arg: None}))
    assert len(calls) == n + 1


def test_gains_and_formats(calls):
    call = lambda **kw: CALLS["norm"][0](**dict(norm_args(), **kw))
    formats = lambda: calls[-1][1][-3]
    call()
    assert formats() == 0 and calls[-1][1][8:10] == (1.0, pytest.approx(1e-5))
    call(q_weight=On(torch.zeros(128)), k_weight=On(torch.zeros(128)), meta_bf16=True)
    assert formats() == saw.SAW_FMT_F32_WEIGHT | saw.SAW_FMT_BF16_META
    call(q_weight=None, k_weight=On(torch.zeros(128)))
    assert formats() == saw.SAW_FMT_F32_WEIGHT
    half = lambda *n: rows(*n, dt=F16)
    call(q=half(3, 4, 128), k=half(3, 2, 128), v=half(3, 2, 128), q_out=half(3, 4, 128), q_weight=half(128), k_weight=None)
    assert formats() == saw.SAW_FMT_F16_INPUT
    refused(calls, "norm", dict(norm_args(), q_weight=half(128)), "q_weight must be 128 contiguous entries")
    refused(calls, "norm", dict(norm_args(), k_weight=rows(64)), "k_weight must be 128")
    refused(calls, "norm", dict(norm_args(), k_weight=On(torch.zeros(256)[::2])), "k_weight must be 128 contiguous")
    refused(calls, "norm", dict(norm_args(), k_weight=On(torch.zeros(128))), "one type")
    CALLS["sparse"][0](**dict(sparse_args(), out=On(torch.zeros(3, 4, 128)), meta_bf16=True))
    assert calls[-1][1][-3] == saw.SAW_FMT_BF16_META
    CALLS["sparse"][0](**sparse_args())
    assert calls[-1][1][-3] == saw.SAW_FMT_OUT_INPUT


@pytest.mark.parametrize("name,kw,text", [
    ("norm", dict(q_out=lambda: rows(3, 5, 128)), "q_out must have q's heads"),
    ("norm", dict(v=lambda: rows(3, 3, 128)), "v must have k's heads"),
    ("norm", dict(num_pages=5), "_cache must have"),
    ("summary", dict(k_cache=lambda: On(cache().t[:-1])), "k_cache must have"),
    ("summary", dict(summary=lambda: On(summary().t[:-1])), "summary must have"),
    ("summary", dict(block_tables=lambda: i32(2, 4)), "block_tables must have 3 rows"),
    ("summary", dict(new_lens=lambda: i32(4)), "new_lens must have 3"),
    ("summary", dict(num_kv_heads=3), "must have"),
    ("select", dict(summary=lambda: On(summary().t[:-1])), "summary must have"),
    ("select", dict(block_tables=lambda: i32(2, 4)), "block_tables must have 3 rows"),
    ("select", dict(seq_lens=lambda: i32(2)), "seq_lens must have 3"),
    ("select", dict(sel_tables=lambda: i32(3, 3, 3)), "sel_tables must be"),
    ("select", dict(sel_tables=lambda: i32(3, 6)), "3 dimensions"),
    ("select", dict(sel_pages=lambda: i32(3, 2, 4)), "sel_pages must be of sel_tables' shape"),
    ("select", dict(sel_lens=lambda: i32(3, 1)), "sel_lens must have 6"),
    ("select", dict(q=lambda: On(torch.zeros(3, 4, 256, dtype=BF)[:, :, ::2])), "q must be contiguous"),
    ("select", dict(q=lambda: On(torch.zeros(3, 4, 128))), "bfloat16 or float16"),
    ("sparse", dict(out=lambda: rows(3, 4, 128, dt=F16)), "float32 or q's type"),
    ("sparse", dict(out=lambda: rows(3, 4, 64)), "of one shape"),
    ("sparse", dict(q=lambda: On(torch.zeros(3, 4, 256, dtype=BF)[:, :, ::2])), "contiguous"),
    ("sparse", dict(sel_tables=lambda: i32(3, 3, 4)), "sel_tables must be"),
    ("sparse", dict(sel_lens=lambda: i32(5)), "sel_lens must have 6"),
    ("sparse", dict(k_cache=lambda: On(cache().t[:-1])), "k_cache must have"),
    ("sparse", dict(v_cache=lambda: On(cache().t[:-1])), "v_cache must have"),
    ("sparse", dict(workspace=lambda: On(torch.zeros(64)[::2])), "workspace must be contiguous"),
])
def test_shapes(calls, name, kw, text):
    refused(calls, name, dict(CALLS[name][1](), **{k: v() if callable(v) else v for k, v in kw.items()}), text)
