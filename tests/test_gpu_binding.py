"""What the Python binding of the serving step's calls refuses before anything
is launched, and the forms of a stream it takes."""
import pytest
import torch

import bit_paged_kv_gb300 as saw

pytestmark = pytest.mark.gpu


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def tables(**kw):
    a = dict(cached_lens=i32(4), new_lens=i32(4), free_pages=i32(8), num_free=i32(1), page_size=16, num_pages=8,
             block_tables=i32(4, 6), seq_lens=i32(4), cu_q_lens=i32(5), slot_mapping=i32(12), positions=i32(12),
             pages_taken=i32(1), src_tables=i32(4, 6), src_rows=i32(4), dev_status=i32(1))
    a.update(kw)
    saw.saw_build_tables(**a)


def rope(dt=torch.bfloat16, **kw):
    z = lambda *s: torch.zeros(s, dtype=dt, device="cuda")
    n = saw.saw_cache_bytes(4, 16, 2, 128)
    c = torch.zeros(n, dtype=torch.uint8, device="cuda")
    a = dict(q=z(3, 4, 128), k=z(3, 2, 128), v=z(3, 2, 128), positions=i32(3), cos_sin=torch.zeros(8, 128, device="cuda"),
             slot_mapping=i32(3) - 1, q_out=z(3, 4, 128), k_cache=c, v_cache=c.clone(), num_pages=4, page_size=16,
             rotate_k=True, rotate_v=True, block_h=128)
    a.update(kw)
    saw.saw_rope_append(**a)


def prefix(**kw):
    n = saw.saw_cache_bytes(4, 16, 2, 128)
    c = torch.zeros(n, dtype=torch.uint8, device="cuda")
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    a = dict(q=q, k_cache=c, v_cache=c, block_tables=i32(3, 4), seq_lens=i32(3), cu_group_seqs=i32(2),
             prefix_lens=i32(1), max_prefix_len=16, max_own_len=16, num_kv_heads=2, num_pages=4, page_size=16,
             rotate_k=True, rotate_v=True, block_h=128, out=torch.empty_like(q))
    a.update(kw)
    saw.saw_prefix_decode_int4(**a)


WIDE = dict(dtype=torch.int64, device="cuda")
BF = dict(dtype=torch.bfloat16, device="cuda")
REFUSED = [
    (tables, dict(new_lens=lambda: torch.zeros(4, **WIDE)), ValueError, "new_lens must be contiguous int32"),
    (tables, dict(new_lens=lambda: torch.zeros(4, dtype=torch.int32)), ValueError, "CUDA device"),
    (tables, dict(new_lens=None), AttributeError, ""),
    (tables, dict(cached_lens=lambda: i32(4, 2)[:, 0]), ValueError, "cached_lens must be contiguous"),
    (tables, dict(seq_lens=(5,)), ValueError, "seq_lens must have 4 entries, not 5"),
    (tables, dict(cu_q_lens=(4,)), ValueError, "cu_q_lens must have 5 entries"),
    (tables, dict(block_tables=(3, 6)), ValueError, "block_tables must have 4 rows, not 3"),
    (tables, dict(block_tables=(24,)), ValueError, "2 dimensions"),
    (tables, dict(positions=(11,)), ValueError, "positions must have 12"),
    (tables, dict(num_free=(2,)), ValueError, "num_free must have 1"),
    (tables, dict(num_pages=1 << 40), OverflowError, ""),
    (tables, dict(page_size=16.0), TypeError, ""),
    (tables, dict(page_size=8), saw.SawError, "SAW_ERR_UNSUPPORTED"),
    (rope, dict(q=lambda: torch.zeros(3, 4, 128, dtype=torch.float16, device="cuda")), ValueError, "q must be"),
    (rope, dict(k=lambda: torch.zeros(3, 2, 128, device="cuda")), ValueError, "bfloat16 or float16"),
    (rope, dict(k=lambda: torch.zeros(3, 256, **BF)), ValueError, "3 dimensions"),
    (rope, dict(v=lambda: torch.zeros(3, 3, 128, **BF)), ValueError, "v must have k's heads"),
    (rope, dict(q_out=lambda: torch.zeros(3, 5, 128, **BF)), ValueError, "q_out must have q's heads"),
    (rope, dict(v=lambda: torch.zeros(3, 2, 256, **BF)[..., ::2]), ValueError, "v must be"),
    (rope, dict(k=lambda: torch.zeros(3, 128, 2, **BF).transpose(1, 2)), ValueError, "k must be"),
    (rope, dict(positions=(4,)), ValueError, "positions must have 3"),
    (rope, dict(slot_mapping=lambda: torch.zeros(3, **WIDE)), ValueError, "slot_mapping must be"),
    (rope, dict(cos_sin=lambda: torch.zeros(8, 128, dtype=torch.float64, device="cuda")), ValueError, "cos_sin must be"),
    (rope, dict(block_h=48), saw.SawError, "SAW_ERR_INVALID_ARG"),
    (prefix, dict(out=lambda: torch.zeros(3, 4, 128, dtype=torch.float16, device="cuda")), ValueError, "out must be"),
    (prefix, dict(out=lambda: torch.zeros(3, 4, 64, **BF)), ValueError, "one shape"),
    (prefix, dict(q=lambda: torch.zeros(4, 3, 128, **BF).transpose(0, 1)), ValueError, "contiguous"),
    (prefix, dict(block_tables=(2, 4)), ValueError, "block_tables must have 3 rows"),
    (prefix, dict(cu_group_seqs=(3,)), ValueError, "cu_group_seqs must have 2"),
    (prefix, dict(seq_lens=(2,)), ValueError, "seq_lens must have 3"),
    (prefix, dict(mode=5), saw.SawError, "SAW_ERR_INVALID_ARG"),
]


@pytest.mark.parametrize("call,kw,error,text", REFUSED, ids=[f"{c.__name__}-{i}" for i, (c, *_) in enumerate(REFUSED)])
def test_refused(call, kw, error, text):
    kw = {k: i32(*v) if isinstance(v, tuple) else v() if callable(v) else v for k, v in kw.items()}
    with pytest.raises(error, match=text or None):
        call(**kw)
    torch.cuda.synchronize()


def test_streams():
    """No stream: the current one; a Stream; a handle."""
    side = torch.cuda.Stream()
    want = None
    for stream in (None, side, side.cuda_stream, 0):
        t = torch.full((40, 32), 9.0, device="cuda")
        torch.cuda.synchronize()
        saw.saw_rope_table(t, stream=stream)
        torch.cuda.synchronize()
        want = t if want is None else want
        assert torch.equal(t, want) and t[0, 0] == 1 and t[0, 16] == 0
    with torch.cuda.stream(side):
        t = torch.full((40, 32), 9.0, device="cuda")
        saw.saw_rope_table(t)
        assert torch.equal(t.cpu(), want.cpu())


def test_calls_that_pass():
    """The arguments the refusals start from, a single token with any stride, and no optional ones."""
    tables()
    tables(cached_lens=None, src_tables=None, src_rows=None, positions=None, pages_taken=None, dev_status=None,
           num_free=None)
    rope()
    rope(dt=torch.float16, q=None, q_out=None)
    rope(v=None, v_cache=None)
    rope(q=torch.zeros(1, 4, 128, **BF).as_strided((1, 4, 128), (7, 128, 1)), k=torch.zeros(1, 2, 128, **BF),
         v=torch.zeros(1, 2, 128, **BF), q_out=torch.zeros(1, 4, 128, **BF), positions=i32(1), slot_mapping=i32(1))
    prefix()
    torch.cuda.synchronize()
