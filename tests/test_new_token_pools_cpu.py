"""Shapes and types of the tensors that the new-token calls take, on the host:
what the binding hands to the C ABI, and what it refuses before."""
import pytest
import torch

from gpu_common import lib

dsa = lib()
BF = torch.bfloat16


def _x(heads, dim, n=3):
    return torch.zeros((n, heads, dim), dtype=BF)


@pytest.mark.parametrize("heads,dim,shape,row,head", [
    (4, 64, (8, 16, 4, 64), 256, 64),
    (4, 64, (8, 16, 4, 80), 320, 80),          # head slots wider than the head
    (4, 64, (8, 16, 6, 64), 384, 64),          # more slots than heads
    (1, 64, (8, 16, 1, 64), 64, 64),
    (4, 64, (8, 16, 256), 256, 64),            # a 3-D pool's heads are packed
    (4, 64, (8, 16, 320), 320, 64),
])
def test_a_part_s_rows_and_heads_lie_where_the_pool_s_shape_says(heads, dim, shape, row, head):
    pool = torch.zeros(shape, dtype=BF)
    parts = dsa.HeadParts([dsa.HeadPart(_x(heads, dim), pool)])
    c = parts.c(True)[0]
    assert (c.out_token_stride, c.out_head_stride) == (row, head)
    assert parts.pool_rows == 8 * 16


@pytest.mark.parametrize("shape", [(8, 16, 2, 128), (8, 16, 4, 56), (8, 16, 3, 64), (8, 16, 1, 256)])
def test_a_pool_whose_heads_do_not_hold_the_part_s_is_refused(shape):
    with pytest.raises(ValueError, match="pool"):
        dsa.HeadParts([dsa.HeadPart(_x(4, 64), torch.zeros(shape, dtype=BF))]).c(True)


# ------------------------------------------------ pools of several heads, read --
def _layout(nb=4, bs=64):
    bt = torch.arange(nb, dtype=torch.int32).reshape(2, nb // 2)
    return dsa.PagedLayout(bt, torch.full((2,), 100, dtype=torch.int32), bs, nb, 128)


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _attention_calls(k, v):
    """Every call that reads K and V pools, on host tensors."""
    lay, ws = _layout(), _z(4096, dtype=torch.uint8)
    q, out, lse = _z(2, 4, 64), _z(2, 4, 64), _z(2, 4, dtype=torch.float32)
    idx, one = _z(2, 8, dtype=torch.int32), _z(2, dtype=torch.int32)
    qi, w, kidx = _z(2, 4, 64), _z(2, 4, dtype=torch.float32), _z(4, 64, 64)
    new = _z(2, 64)
    sc = _z(2, 128, dtype=torch.float32)
    step = (new, k, new, kidx, qi, w, q, 8, 0.1)
    return {
        "prefix_attn_decode": lambda: dsa.prefix_attn_decode(lay, q, k, v, 0, 0.1, out, lse, ws),
        "sparse_attn_decode": lambda: dsa.sparse_attn_decode(lay, q, k, v, idx, 0.1, out, lse, ws),
        "sparse_attn_prefill": lambda: dsa.sparse_attn_prefill(lay, q, k, v, idx, 0.1, out, lse, ws,
                                                               q_seq=one, q_pos=one),
        "decode_step": lambda: dsa.decode_step(lay, *step, sc, idx, out, lse, ws, v_new=new, v_pool=v),
        "prefill_step": lambda: dsa.prefill_step(lay, 0, one, one, *step, sc, idx, out, lse, ws,
                                                 v_new=new, v_pool=v),
        "prefill_step_chunked": lambda: dsa.prefill_step_chunked(lay, 0, one, one, *step, 128, idx, out,
                                                                 lse, ws, v_new=new, v_pool=v),
        "cache_write": lambda: dsa.cache_write(lay, one, one, ws, kv_new=new, kv_pool=k),
    }


CALLS = list(_attention_calls(None, None))


@pytest.mark.parametrize("call", CALLS)
def test_a_pool_of_several_heads_is_not_read_as_rows_of_one(call):
    """The calls read one row of a position per pool; the last dimension of
    [num_blocks, block_size, heads, dim] is a head, not a row."""
    one, four = _z(4, 64, 64), _z(4, 64, 4, 64)
    with pytest.raises(ValueError, match="heads"):
        _attention_calls(four, one)[call]()
    if call != "cache_write":
        with pytest.raises(ValueError, match="heads"):
            _attention_calls(one, four)[call]()


@pytest.mark.parametrize("call", CALLS)
def test_pools_of_one_head_are_taken_with_and_without_the_dimension(call):
    """... up to the check that host tensors stop at."""
    for k in (_z(4, 64, 64), _z(4, 64, 1, 64), _z(256, 64)):
        with pytest.raises(ValueError, match="CUDA"):
            _attention_calls(k, k)[call]()


# ------------------------------------------------------------- pages of one row --
@pytest.mark.parametrize("make", [
    lambda: _z(1, 8, 256).transpose(0, 1),                       # strides (256, 2048, 1)
    lambda: _z(8, 256).as_strided((8, 1, 256), (256, 8, 1)),     # (256, 8, 1)
    lambda: _z(1, 8, 4, 64).transpose(0, 1),
], ids=["transposed", "as-strided", "with-heads"])
def test_pages_of_one_row_may_carry_any_stride(make):
    pool = make()
    assert pool.shape[:2] == (8, 1) and pool.is_contiguous()
    parts = dsa.HeadParts([dsa.HeadPart(_x(4, 64), pool)])
    c = parts.c(True)[0]
    assert (c.out_token_stride, c.out_head_stride, parts.pool_rows) == (256, 64, 8)


# ---------------------------------------------------------------- operand types --
@pytest.mark.parametrize("name,dtype", [("q", torch.float16), ("q", torch.int16), ("k_pool", torch.float16),
                                        ("v_pool", torch.float16), ("out", torch.float16),
                                        ("lse", torch.int32), ("ws", torch.float32)])
def test_the_attention_refuses_operands_of_another_type_of_the_same_size(name, dtype):
    a = dict(q=_z(2, 4, 64), k_pool=_z(4, 64, 64), v_pool=_z(4, 64, 64), out=_z(2, 4, 64),
             lse=_z(2, 4, dtype=torch.float32), ws=_z(4096, dtype=torch.uint8))
    a[name] = a[name].to(dtype)
    with pytest.raises(TypeError, match=name):
        dsa.prefix_attn_decode(_layout(), a["q"], a["k_pool"], a["v_pool"], 0, 0.1, a["out"], a["lse"],
                               a["ws"])


@pytest.mark.parametrize("name", ["seq", "pos"])
def test_the_appends_refuse_positions_that_are_not_int32(name):
    a = dict(seq=_z(3, dtype=torch.int32), pos=_z(3, dtype=torch.int32))
    a[name] = a[name].float()
    with pytest.raises(TypeError, match=name):
        dsa.cache_append(_layout(), a["seq"], a["pos"], [dsa.HeadPart(_x(1, 64), _z(4, 64, 64))],
                         _z(4096, dtype=torch.uint8))
    if name == "pos":
        with pytest.raises(TypeError, match=name):
            dsa.head_norm_rope([dsa.HeadPart(_x(1, 64), _x(1, 64))], a["pos"])


def _index_calls(kidx):
    """Every call that reads or writes an indexer-key pool, on host tensors."""
    lay, ws = _layout(), _z(4096, dtype=torch.uint8)
    qi, w, one = _z(2, 4, 64), _z(2, 4, dtype=torch.float32), _z(2, dtype=torch.int32)
    sc, idx, bound = _z(2, 128, dtype=torch.float32), _z(2, 8, dtype=torch.int32), _z(4, 2, 64)
    q, out, lse, new, kv = _z(2, 4, 64), _z(2, 4, 64), _z(2, 4, dtype=torch.float32), _z(2, 64), _z(4, 64, 64)
    step = (new, kv, new, kidx, qi, w, q, 8, 0.1)
    return {
        "index_score": lambda: dsa.index_score(lay, qi, w, kidx, sc, ws),
        "index_score_prefill": lambda: dsa.index_score_prefill(lay, 0, qi, w, kidx, sc, ws),
        "index_bounds_update": lambda: dsa.index_bounds_update(lay, kidx, bound, ws),
        "index_score_bounded": lambda: dsa.index_score_bounded(lay, qi, w, kidx, bound, 8, sc, ws),
        "decode_step": lambda: dsa.decode_step(lay, *step, sc, idx, out, lse, ws),
        "prefill_step": lambda: dsa.prefill_step(lay, 0, one, one, *step, sc, idx, out, lse, ws),
        "prefill_step_chunked": lambda: dsa.prefill_step_chunked(lay, 0, one, one, *step, 128, idx, out,
                                                                 lse, ws),
        "cache_write": lambda: dsa.cache_write(lay, one, one, ws, kidx_new=new, kidx_pool=kidx),
    }


@pytest.mark.parametrize("call", list(_index_calls(None)))
def test_an_indexer_key_pool_of_several_heads_is_refused_too(call):
    with pytest.raises(ValueError, match="heads"):
        _index_calls(_z(4, 64, 2, 64))[call]()
    for k in (_z(4, 64, 64), _z(4, 64, 1, 64), _z(256, 64)):
        with pytest.raises(ValueError, match="CUDA"):
            _index_calls(k)[call]()
