"""Host-only checks of the batched operators: what their entry points refuse,
before any GPU is touched (addresses are never followed here), and the rotary
frequencies, which are host work."""

import pytest

pytest.importorskip("torch")

A = 0x100000  # aligned addresses, apart from one another
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def mk():
    import __graft_entry__
    import os
    if not os.path.exists(__graft_entry__.LIB):
        __graft_entry__.build()
    from moe_decode_layer_persistent_gb300 import binding
    return binding


def refused(mk, call, status):
    with pytest.raises(mk.MkError) as e:
        call()
    assert e.value.status == status, e.value


def slots_io(mk, **over):
    f = dict(n_requests=4, n_rows=16, page_size=16, max_pages=8, table_stride=8, n_pages=64,
             n_free=32, prefix_len=0, cached_lens=A, new_lens=2 * A, free_pages=3 * A,
             free_head=4 * A, block_table=5 * A, cu_rows=6 * A, lens=7 * A, positions=8 * A,
             slots=9 * A, row_request=10 * A, summary=11 * A)
    f.update(over)
    return mk.mk_slots_io(**f)


@pytest.mark.parametrize("over", [
    dict(n_requests=-1), dict(n_requests=65537), dict(n_rows=-1), dict(page_size=0),
    dict(max_pages=-1), dict(n_pages=-1), dict(n_free=-1), dict(prefix_len=-1),
    dict(table_stride=7), dict(max_pages=1 << 28, table_stride=1 << 28),
    dict(max_pages=1 << 26, table_stride=1 << 26, prefix_len=(1 << 30) + 1),
    dict(cached_lens=0), dict(new_lens=0), dict(lens=0), dict(cu_rows=0), dict(summary=0),
    dict(block_table=0), dict(positions=0), dict(slots=0), dict(free_pages=0),
    dict(cached_lens=A + 2), dict(slots=9 * A + 4), dict(summary=11 * A + 1),
    dict(lens=A), dict(summary=4 * A), dict(lens=A + 12), dict(positions=8 * A, slots=8 * A),
    dict(block_table=3 * A + 64), dict(cu_rows=7 * A + 8)])
def test_slots_refusals(mk, over):
    refused(mk, lambda: mk.mk_build_slots(slots_io(mk, **over)), INVALID)


def test_null_arguments(mk):
    for call in (lambda: mk._check("f", mk._lib_mk_build_slots(None, None)),
                 lambda: mk._check("f", mk._lib_mk_rope_create(None, mk._vp())),
                 lambda: mk._check("f", mk._lib_mk_rope_apply(None, rope_io(mk), None)),
                 lambda: mk._check("f", mk._lib_mk_prefix_attn(None, 16 * A, 1 << 30, None)),
                 lambda: mk._check("f", mk._lib_mk_prefix_attn_workspace(None, mk._i64()))):
        refused(mk, call, INVALID)
    assert mk.mk_prefix_attn_status(None) == INVALID
    mk.mk_rope_destroy(None)


@pytest.mark.parametrize("over,status", [
    (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=100), UNSUPPORTED),
    (dict(head_dim=264), UNSUPPORTED), (dict(rot_dim=0), INVALID), (dict(rot_dim=136), INVALID),
    (dict(rot_dim=24), UNSUPPORTED), (dict(rot_dim=12, layout="interleaved"), UNSUPPORTED),
    (dict(theta=0.5), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(factor=2.0), INVALID), (dict(scaling="linear", factor=0.5), INVALID),
    (dict(scaling="linear", factor=float("inf")), INVALID),
    (dict(scaling="parts", factor=2.0), INVALID),
    (dict(scaling="parts", factor=2.0, orig_ctx=4096, beta_fast=1.0, beta_slow=2.0), INVALID),
    (dict(attn_factor=-1.0), INVALID)])
def test_rope_config_refusals(mk, over, status):
    cfg = dict(head_dim=128)
    cfg.update(over)
    refused(mk, lambda: mk.mk_rope_create(mk.make_rope_config(**cfg)), status)


def test_rope_config_unknown_choices(mk):
    for field in ("layout", "scaling"):
        for value in (-1, 4):
            c = mk.make_rope_config(128)
            setattr(c, field, value)
            refused(mk, lambda: mk.mk_rope_create(c), INVALID)


def rope_io(mk, **over):
    f = dict(n_rows=4, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=0, q=A, q_stride=1536,
             q_out=2 * A, q_out_stride=1024, k=A + 2048, k_stride=1536, v=A + 2560, v_stride=1536,
             positions=3 * A, slots=4 * A, k_cache=5 * A, v_cache=6 * A, n_slots=64)
    f.update(over)
    return mk.mk_rope_io(**f)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(head_dim=64), INVALID),
    (dict(n_rows=-1), INVALID), (dict(n_q_heads=0), INVALID), (dict(q=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=5000, q_stride=640000, q_out_stride=640000), UNSUPPORTED),
    (dict(q_out=0), INVALID), (dict(slots=0), INVALID), (dict(k_cache=0), INVALID),
    (dict(v_cache=0), INVALID), (dict(positions=0), INVALID), (dict(n_slots=-1), INVALID),
    (dict(q=A + 8), INVALID), (dict(v_cache=6 * A + 2), INVALID), (dict(slots=4 * A + 4), INVALID),
    (dict(q_stride=1016), INVALID), (dict(q_stride=1028), INVALID), (dict(k_stride=248), INVALID),
    (dict(v_stride=1537), INVALID), (dict(q_out=A + 1024), INVALID),
    (dict(q_out=A, q_out_stride=1024), INVALID), (dict(positions=2 * A), INVALID),
    (dict(slots=2 * A + 64), INVALID)])
def test_rope_refusals(mk, over, status):
    r = mk.mk_rope_create(mk.make_rope_config(128))
    try:
        refused(mk, lambda: mk.mk_rope_apply(r, rope_io(mk, **over)), status)
        mk.mk_rope_apply(r, rope_io(mk, n_rows=0))  # nothing to do, on any machine
    finally:
        mk.mk_rope_destroy(r)


def attn_io(mk, **over):
    f = dict(n_requests=4, n_rows=8, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=0,
             page_size=16, n_pages=64, prefix_len=100, max_pages=8, table_stride=8, window=0,
             scale=0.0, q=A, q_stride=1024, k_cache=2 * A, v_cache=3 * A, prefix_pages=4 * A,
             block_table=5 * A, lens=6 * A, cu_rows=7 * A, tree_mask=0, out=8 * A,
             out_stride=1024, lse=9 * A)
    f.update(over)
    return mk.mk_prefix_attn_io(**f)


def attn(mk, io, workspace=16 * A, size=1 << 40):
    mk._check("mk_prefix_attn", mk._lib_mk_prefix_attn(io, workspace, size, None))


@pytest.mark.parametrize("over,status", [
    (dict(n_requests=0), INVALID), (dict(n_requests=65537), INVALID), (dict(n_rows=-1), INVALID),
    (dict(n_q_heads=7), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_q_heads=0), INVALID),
    (dict(n_q_heads=130, q_stride=1 << 15, out_stride=1 << 15), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=1 << 17), UNSUPPORTED), (dict(n_pages=-1), INVALID),
    (dict(n_pages=1 << 27), INVALID), (dict(prefix_len=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(table_stride=7), INVALID), (dict(max_pages=1 << 27, table_stride=1 << 27), INVALID),
    (dict(n_requests=65536, n_rows=65536, max_pages=1 << 20, table_stride=1 << 20), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(window=63, tree_mask=10 * A), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=3e38), INVALID), (dict(q=0), INVALID), (dict(out=0), INVALID),
    (dict(out=A), INVALID), (dict(k_cache=0), INVALID), (dict(v_cache=0), INVALID),
    (dict(lens=0), INVALID), (dict(cu_rows=0), INVALID), (dict(block_table=0), INVALID),
    (dict(prefix_pages=0), INVALID), (dict(q_stride=1020), INVALID), (dict(q_stride=1016), INVALID),
    (dict(out_stride=1028), INVALID), (dict(q=A + 8), INVALID), (dict(out=8 * A + 2), INVALID),
    (dict(k_cache=2 * A + 8), INVALID), (dict(lens=6 * A + 2), INVALID),
    (dict(tree_mask=10 * A + 4), INVALID), (dict(lse=9 * A + 2), INVALID)])
def test_attention_refusals(mk, over, status):
    refused(mk, lambda: attn(mk, attn_io(mk, **over)), status)


def test_attention_workspace_refusals(mk):
    refused(mk, lambda: attn(mk, attn_io(mk), workspace=0), INVALID)
    refused(mk, lambda: attn(mk, attn_io(mk), workspace=16 * A + 128), INVALID)
    refused(mk, lambda: mk._check("f", mk._lib_mk_prefix_attn_workspace(attn_io(mk), None)), INVALID)


def test_binding_refuses_what_the_library_would_misread(mk):
    import torch
    t = torch.zeros(4, dtype=torch.int32)           # host memory
    q = torch.zeros(2, 2, 16, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, 2, 16, dtype=torch.bfloat16)
    refused(mk, lambda: mk.make_slots_io(t, t, t, None, t[None], t, t, t, t.long(), None, t, 16, 8), INVALID)
    refused(mk, lambda: mk.make_rope_io(q, q, q, q, t, t.long(), pool, pool), INVALID)
    refused(mk, lambda: mk.make_rope_io(None, None, None, None, t, t, None, None), INVALID)
    refused(mk, lambda: mk.make_rope_io(q[0], q, None, None, t, t, None, None), INVALID)
    refused(mk, lambda: mk.make_prefix_attn_io(q, pool, pool, q, t, t, t[None], t, 4), INVALID)
    # one thing at a time, with the device taken as given
    refused(mk, lambda: mk._vec("f", t, torch.int64, -1), INVALID)
    refused(mk, lambda: mk._vec("f", t, torch.int32, 0), INVALID)
    refused(mk, lambda: mk._vec("f", t, torch.int32, -1, 5), INVALID)
    refused(mk, lambda: mk._vec("f", t[::2], torch.int32, -1), INVALID)
    refused(mk, lambda: mk._rows("f", q.transpose(0, 1), (2, 2, 16), q.dtype, -1), INVALID)
    refused(mk, lambda: mk._rows("f", q, (2, 2, 32), q.dtype, -1), INVALID)
    refused(mk, lambda: mk._rows("f", q.half(), (2, 2, 16), q.dtype, -1), INVALID)
    refused(mk, lambda: mk._table("f", t.repeat(4, 1).t(), torch.int32, -1), INVALID)
    refused(mk, lambda: mk._table("f", t, torch.int32, -1), INVALID)
    refused(mk, lambda: mk._kind("f", torch, torch.zeros(1)), INVALID)
    assert mk._vec("f", None, torch.int32, 0) == 0
    assert mk._rows("f", q[:, :1], (2, 1, 16), q.dtype, -1) == (q.data_ptr(), 32)


def test_packed_fields_are_the_structs(mk):
    """The packed layouts are those of the ctypes structs, field by field."""
    import struct
    for cls, fmt in ((mk.mk_slots_io, "@4iqiii11P"), (mk.mk_rope_io, "@5iPqPqPqPqPPPPq"),
                     (mk.mk_prefix_attn_io, "@10iqifPqPPPPPPPPqP")):
        values = [i + 1 for i in range(len(cls._fields_))]
        got = cls.from_buffer_copy(struct.Struct(fmt).pack(*values))
        assert [getattr(got, f) for f, _ in cls._fields_] == values


@pytest.mark.parametrize("make", [
    lambda t: t[:8].expand(4, 8), lambda t: t.as_strided((4, 8), (3, 1)), lambda t: t[:1].expand(4, 1),
    lambda t: t.as_strided((4, 8), (7, 1))])
def test_tables_whose_rows_overlap(mk, make):
    """Rows that share memory keep their stride, which the library refuses: a
    stride of its own would lead it behind the table."""
    import torch
    table = make(torch.zeros(64, dtype=torch.int32))
    _, rows, cols, stride = mk._table("f", table, torch.int32, -1)
    assert (rows, cols, stride) == (*table.shape, table.stride(0))
    refused(mk, lambda: attn(mk, attn_io(mk, max_pages=cols, table_stride=stride)), INVALID)
    refused(mk, lambda: mk.mk_build_slots(slots_io(mk, max_pages=cols, table_stride=stride)), INVALID)


def test_tables_of_one_row_or_column(mk):
    """A single row has no stride to respect; a table's rows may have gaps."""
    import torch
    t = torch.zeros(64, dtype=torch.int32)
    assert mk._table("f", t[None], torch.int32, -1)[1:] == (1, 64, 64)
    assert mk._table("f", t[:8].expand(1, 8), torch.int32, -1)[1:] == (1, 8, 8)
    assert mk._table("f", t.as_strided((1, 8), (2, 1)), torch.int32, -1)[1:] == (1, 8, 8)
    assert mk._table("f", t.view(8, 8)[:, :5], torch.int32, -1)[1:] == (8, 5, 8)
    assert mk._table("f", t.view(8, 8)[:, 3:4], torch.int32, -1)[1:] == (8, 1, 8)
    assert mk._table("f", t.view(8, 8)[:, :0], torch.int32, -1)[1:] == (8, 0, 8)
    assert mk._table("f", t[:0].view(0, 8), torch.int32, -1)[1:] == (0, 8, 8)


def test_workspace_refusals_of_the_binding(mk):
    """A workspace is one stretch of memory, on the device of the tensors it is
    for: its address and its number of values do not tell."""
    import torch
    room = torch.zeros(1 << 16, dtype=torch.uint8)
    room = room[-room.data_ptr() % 256:]            # aligned as a workspace has to be
    for bad in (room[:1].expand(1 << 30), room[::2], room[:1 << 14].view(128, 128).t()):
        refused(mk, lambda: mk.mk_prefix_attn(attn_io(mk), bad), INVALID)
    io = attn_io(mk)
    io.device = 1                                   # as make_prefix_attn_io leaves it
    refused(mk, lambda: mk.mk_prefix_attn(io, room), INVALID)


@pytest.mark.parametrize("over,args,status", [
    ({}, (0, 1, 0), INVALID), ({}, (2 * 10 ** 9 + 1, 1, 0), INVALID), ({}, (10 ** 6, 5, 0), INVALID),
    ({}, (10 ** 6, -1, 0), INVALID), ({}, (10 ** 6, 1, -1), INVALID),
    (dict(dtype=1), (10 ** 6, 1, 0), UNSUPPORTED), ({}, (10 ** 6, 1, 0), UNSUPPORTED),   # head_dim 128
    (dict(head_dim=64, lens=0), (10 ** 6, 1, 0), INVALID)])
def test_attention_waits_selftest_refusals(mk, over, args, status):
    assert mk._lib_mk_selftest_attn_waits(attn_io(mk, **over), 16 * A, 1 << 40, *args, None) == status
    assert mk._lib_mk_selftest_attn_waits(None, 16 * A, 1 << 40, 10 ** 6, 1, 0, None) == INVALID


def test_rope_without_rows(mk):
    """Tensors without rows have no address; what does not depend on rows is still checked."""
    r = mk.mk_rope_create(mk.make_rope_config(128))
    empty = dict(n_rows=0, q=0, q_out=0, k=0, v=0, positions=0, slots=0)
    try:
        mk.mk_rope_apply(r, rope_io(mk, **empty))
        mk.mk_rope_apply(r, rope_io(mk, **empty, q_stride=0, q_out_stride=0, k_stride=0, v_stride=0))
        mk.mk_rope_apply(r, rope_io(mk, **empty, n_kv_heads=0, k_cache=0, v_cache=0, n_slots=0))
        for over, status in ((dict(dtype=2), UNSUPPORTED), (dict(head_dim=64), INVALID),
                             (dict(n_q_heads=-1), INVALID), (dict(n_kv_heads=5000), UNSUPPORTED)):
            refused(mk, lambda: mk.mk_rope_apply(r, rope_io(mk, **empty, **over)), status)
    finally:
        mk.mk_rope_destroy(r)
