"""What the Python binding of the serving step's calls checks, on the CPU: the
extension is pointed at entry points that only note their arguments, and at
tensors that claim a device.  Every tensor argument has to be on the call's
device, the caches have to be contiguous and of the size that the call's
counts give, and nothing is called otherwise."""
import ctypes as C

import pytest
import torch

import bit_paged_kv_gb300 as saw
from bit_paged_kv_gb300 import build as saw_build

HERE = 2  # the current device of these tests


class On:
    """A CPU tensor that says it is on a CUDA device."""

    def __init__(self, t, dev=HERE):
        self.t, self.dev = t, dev

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.dev


@pytest.fixture(scope="module")
def calls():
    saw_build.build()
    L, seen = saw.lib(), []
    m = saw._binding._bind_step()
    fakes = []
    for name in ("saw_build_tables", "saw_rope_table", "saw_rope_append", "saw_prefix_decode_int4"):
        f = C.CFUNCTYPE(C.c_int32, *getattr(L, name).argtypes)(lambda *a, name=name: seen.append((name, a)) or 0)
        fakes.append(f)
    at = [C.cast(f, C.c_void_p).value for f in (*fakes, L.saw_cache_bytes)]
    m.init(*at, torch.int32, torch.float32, torch.bfloat16, torch.float16, lambda: HERE, lambda dev: 77)
    yield seen
    saw._binding._bind_step()  # the library's entry points again


def i32(*n):
    return On(torch.zeros(n, dtype=torch.int32))


def rows(*n, dt=torch.bfloat16):
    return On(torch.zeros(n, dtype=dt))


def cache(pages=4, hkv=2, d=128):
    return On(torch.zeros(pages * hkv * 16 * (d // 2 + 4), dtype=torch.uint8))


def tables_args():
    return dict(cached_lens=i32(4), new_lens=i32(4), free_pages=i32(8), num_free=i32(1), page_size=16, num_pages=8,
                block_tables=i32(4, 6), seq_lens=i32(4), cu_q_lens=i32(5), slot_mapping=i32(12), positions=i32(12),
                pages_taken=i32(1), src_tables=i32(4, 6), src_rows=i32(4), dev_status=i32(1))


def table_args():
    return dict(cos_sin=On(torch.zeros(8, 128)))


def rope_args():
    return dict(q=rows(3, 4, 128), k=rows(3, 2, 128), v=rows(3, 2, 128), positions=i32(3),
                cos_sin=On(torch.zeros(8, 128)), slot_mapping=i32(3), q_out=rows(3, 4, 128), k_cache=cache(),
                v_cache=cache(), num_pages=4, page_size=16, rotate_k=True, rotate_v=True, block_h=128,
                dev_status=i32(1))


def prefix_args():
    return dict(q=rows(3, 4, 128), k_cache=cache(), v_cache=cache(), block_tables=i32(3, 4), seq_lens=i32(3),
                cu_group_seqs=i32(2), prefix_lens=i32(1), max_prefix_len=16, max_own_len=16, num_kv_heads=2,
                num_pages=4, page_size=16, rotate_k=True, rotate_v=True, block_h=128, out=rows(3, 4, 128),
                workspace=On(torch.zeros(64, dtype=torch.uint8)), dev_status=i32(1))


CALLS = {"tables": (saw.saw_build_tables, tables_args), "table": (saw.saw_rope_table, table_args),
         "rope": (saw.saw_rope_append, rope_args), "prefix": (saw.saw_prefix_decode_int4, prefix_args)}
TENSORS = [(c, k) for c, (_, args) in CALLS.items() for k, v in args().items() if isinstance(v, On)]


def refused(calls, name, args, text):
    n = len(calls)
    with pytest.raises(ValueError, match=text):
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


@pytest.mark.parametrize("name", ["rope", "prefix"])
@pytest.mark.parametrize("arg", ["k_cache", "v_cache"])
def test_a_cache_that_does_not_hold_the_pages_is_refused(calls, name, arg):
    args = CALLS[name][1]()
    refused(calls, name, dict(args, **{arg: On(args[arg].t[:-1])}), f"{arg} must have {args[arg].numel()} bytes")
    refused(calls, name, dict(args, num_pages=5), "_cache must have")
    wide = On(torch.zeros(args[arg].numel() * 2, dtype=torch.uint8)[::2])
    refused(calls, name, dict(args, **{arg: wide}), f"{arg} must be contiguous")
    bare = On(torch.zeros(1, dtype=torch.uint8).expand(args[arg].numel()))
    refused(calls, name, dict(args, **{arg: bare}), f"{arg} must be contiguous")
    n = len(calls)  # of another type, or larger: fine
    CALLS[name][0](**dict(args, **{arg: On(torch.zeros(args[arg].numel(), dtype=torch.int32))}))
    assert len(calls) == n + 1


def test_workspace_and_status(calls):
    args = prefix_args()
    refused(calls, "prefix", dict(args, workspace=On(torch.zeros(64)[::2])), "workspace must be contiguous")
    CALLS["prefix"][0](**dict(args, workspace=None))
    for name in ("tables", "rope", "prefix"):
        refused(calls, name, dict(CALLS[name][1](), dev_status=i32(0)), "dev_status must have an entry")
        CALLS[name][0](**dict(CALLS[name][1](), dev_status=i32(3)))
        CALLS[name][0](**dict(CALLS[name][1](), dev_status=None))
