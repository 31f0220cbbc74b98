"""Host-only checks of the attention half over a cache in 4 bits: what its entry
points refuse, before any GPU is touched (addresses are never followed here), and
rules read from the sources."""

import pytest

import test_batch_sources as sources
from test_batch_refusals import A, INVALID, UNSUPPORTED, mk, refused  # noqa: F401


def pools(mk, **over):
    f = dict(n_pages=64, page_size=16, n_kv_heads=2, head_dim=128, k_codes=32 * A, k_scales=34 * A, v_codes=36 * A,
             v_scales=38 * A, k_exp=40 * A, v_exp=41 * A)
    f.update(over)
    return mk.mk_kvq_cache(**f)


POOLS = [
    (dict(n_pages=-1), INVALID), (dict(n_pages=1 << 27), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=1 << 17), UNSUPPORTED), (dict(n_kv_heads=0), INVALID),
    (dict(n_kv_heads=5000), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=24), UNSUPPORTED),
    (dict(head_dim=272), UNSUPPORTED), (dict(k_codes=0), INVALID), (dict(v_scales=0), INVALID),
    (dict(k_codes=32 * A + 8), INVALID), (dict(v_scales=38 * A + 1), INVALID), (dict(k_exp=40 * A + 2), INVALID)]


# ----------------------------------------------------------------- append

def append_io(mk, kvq=None, **over):
    f = dict(n_rows=4, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=0, bits=4, eps=1e-6, q=A, q_stride=1536,
             q_out=2 * A, q_out_stride=1024, k=A + 2048, k_stride=1536, v=A + 2560, v_stride=1536, positions=3 * A,
             slots=4 * A, q_norm=5 * A, k_norm=6 * A, k_cache=7 * A, v_cache=8 * A, n_slots=64,
             kvq=kvq if kvq is not None else pools(mk))
    f.update(over)
    return mk.mk_qkv_append_io(**f)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(bits=8), UNSUPPORTED), (dict(n_rows=-1), INVALID), (dict(n_q_heads=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(head_dim=64), INVALID), (dict(head_dim=264), UNSUPPORTED),
    (dict(head_dim=100), UNSUPPORTED), (dict(n_q_heads=5000), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(q=0), INVALID), (dict(q_out=0), INVALID),
    (dict(k=0), INVALID), (dict(slots=0), INVALID), (dict(positions=0), INVALID), (dict(q=A + 8), INVALID),
    (dict(q_norm=5 * A + 2), INVALID), (dict(k_norm=6 * A + 8), INVALID), (dict(slots=4 * A + 4), INVALID),
    (dict(q_stride=1016), INVALID), (dict(k_stride=252), INVALID), (dict(v_stride=1537), INVALID),
    (dict(q_out_stride=1020), INVALID), (dict(q_out=A + 1024), INVALID), (dict(q_out=A, q_out_stride=1024), INVALID),
    (dict(positions=2 * A), INVALID), (dict(slots=2 * A + 64), INVALID), (dict(q_norm=2 * A + 64), INVALID),
    (dict(k=32 * A), INVALID), (dict(v=36 * A + 64), INVALID), (dict(q_out=34 * A), INVALID),
    (dict(positions=38 * A), INVALID), (dict(bits=16, k_cache=0), INVALID), (dict(bits=16, v_cache=0), INVALID),
    (dict(bits=16, n_slots=-1), INVALID), (dict(bits=16, k_cache=7 * A + 4), INVALID)])
def test_append_refusals(mk, over, status):
    r = mk.mk_rope_create(mk.make_rope_config(128))
    try:
        refused(mk, lambda: mk.mk_qkv_append(r, append_io(mk, **over)), status)
    finally:
        mk.mk_rope_destroy(r)


@pytest.mark.parametrize("over,status", POOLS + [
    (dict(n_kv_heads=4), INVALID), (dict(head_dim=64), INVALID), (dict(v_codes=32 * A + 64), INVALID),
    (dict(k_scales=32 * A), INVALID), (dict(v_exp=32 * A), INVALID)])
def test_append_pool_refusals(mk, over, status):
    refused(mk, lambda: mk.mk_qkv_append(None, append_io(mk, pools(mk, **over))), status)


def test_append_without_rows(mk):
    empty = dict(n_rows=0, q=0, q_out=0, k=0, v=0, positions=0, slots=0)
    mk.mk_qkv_append(None, append_io(mk, **empty))
    mk.mk_qkv_append(None, append_io(mk, **empty, n_kv_heads=0, kvq=pools(mk, n_pages=-1)))
    refused(mk, lambda: mk.mk_qkv_append(None, append_io(mk, **empty, dtype=3)), UNSUPPORTED)
    refused(mk, lambda: mk.mk_qkv_append(None, append_io(mk, **empty, kvq=pools(mk, page_size=4))), UNSUPPORTED)


def test_append_takes_rows_of_one_projection(mk):
    """k and v between the rows of q_out, as in place in a projection's output: nothing
    to refuse (what follows is the GPU's absence or presence)."""
    io = append_io(mk, q_out=A, q_out_stride=1536)
    try:
        mk._check("f", mk._lib_mk_qkv_append(None, io, None))
    except mk.MkError as e:
        assert e.status != UNSUPPORTED


# ------------------------------------------------------------------- read

@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(n_rows=-1), INVALID), (dict(n_rows=1025, slots=0), INVALID),
    (dict(k_out=0, v_out=0), INVALID), (dict(k_out=A + 8), INVALID), (dict(slots=3 * A + 4), INVALID),
    (dict(v_out=A + 512), INVALID), (dict(k_out=32 * A), INVALID), (dict(v_out=38 * A), INVALID),
    (dict(k_out=3 * A), INVALID), (dict(k_out=40 * A), INVALID)])
def test_read_refusals(mk, over, status):
    f = dict(kvq=pools(mk), n_rows=8, dtype=0, slots=3 * A, k_out=A, v_out=2 * A)
    f.update(over)
    refused(mk, lambda: mk.mk_kvq_read(mk.mk_kvq_read_io(**f)), status)


@pytest.mark.parametrize("over,status", POOLS)
def test_read_pool_refusals(mk, over, status):
    io = mk.mk_kvq_read_io(kvq=pools(mk, **over), n_rows=8, dtype=0, slots=3 * A, k_out=A, v_out=2 * A)
    refused(mk, lambda: mk.mk_kvq_read(io), status)


def test_read_without_rows(mk):
    mk.mk_kvq_read(mk.mk_kvq_read_io(kvq=pools(mk), n_rows=0, dtype=1))


# -------------------------------------------------------------- attention

def attn_io(mk, kvq=None, **over):
    f = dict(n_requests=4, n_rows=8, n_q_heads=8, dtype=0, max_pages=8, window=0, scale=0.0, table_stride=8,
             kvq=kvq if kvq is not None else pools(mk), q=A, q_stride=1024, block_table=5 * A, lens=6 * A,
             cu_rows=7 * A, tree_mask=0, out=8 * A, out_stride=1024, lse=9 * A)
    f.update(over)
    return mk.mk_kvq_attn_io(**f)


def attn(mk, io, workspace=64 * A, size=1 << 30):
    mk._check("mk_kvq_attn", mk._lib_mk_kvq_attn(io, workspace, size, None))


@pytest.mark.parametrize("over,status", [
    (dict(n_requests=0), INVALID), (dict(n_requests=65537), INVALID), (dict(n_rows=-1), INVALID),
    (dict(n_q_heads=7), INVALID), (dict(n_q_heads=0), INVALID),
    (dict(n_q_heads=130, q_stride=1 << 15, out_stride=1 << 15), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(max_pages=-1), INVALID), (dict(table_stride=7), INVALID), (dict(max_pages=1 << 27, table_stride=1 << 27), INVALID),
    (dict(window=-1), INVALID), (dict(window=63, tree_mask=10 * A), UNSUPPORTED), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=0), INVALID), (dict(out=0), INVALID),
    (dict(out=A), INVALID), (dict(out=A + 1024), INVALID), (dict(lens=0), INVALID), (dict(cu_rows=0), INVALID),
    (dict(block_table=0), INVALID), (dict(q_stride=1020), INVALID), (dict(q_stride=1016), INVALID),
    (dict(out_stride=1028), INVALID), (dict(q=A + 8), INVALID), (dict(out=8 * A + 2), INVALID),
    (dict(lens=6 * A + 2), INVALID), (dict(tree_mask=10 * A + 4), INVALID), (dict(lse=9 * A + 2), INVALID),
    (dict(out=32 * A), INVALID), (dict(lse=38 * A), INVALID), (dict(lse=6 * A), INVALID), (dict(out=5 * A), INVALID),
    (dict(lse=8 * A + 64), INVALID), (dict(n_rows=1 << 28, q_stride=1024), UNSUPPORTED)])
def test_attention_refusals(mk, over, status):
    refused(mk, lambda: attn(mk, attn_io(mk, **over)), status)


@pytest.mark.parametrize("over,status", POOLS + [
    (dict(head_dim=96), UNSUPPORTED), (dict(n_kv_heads=3), INVALID),
    (dict(n_kv_heads=4, n_pages=1, page_size=65536, head_dim=128), None)])
def test_attention_pool_refusals(mk, over, status):
    if status is not None:
        refused(mk, lambda: attn(mk, attn_io(mk, pools(mk, **over))), status)


def test_attention_pages_of_two_gigabytes(mk):
    kvq = pools(mk, n_kv_heads=1024, n_pages=1, page_size=65536)
    refused(mk, lambda: attn(mk, attn_io(mk, kvq, n_q_heads=1024, q_stride=1 << 17, out_stride=1 << 17)), UNSUPPORTED)


def test_workspaces(mk):
    import torch
    io = attn_io(mk)
    refused(mk, lambda: attn(mk, io, workspace=0), INVALID)
    refused(mk, lambda: attn(mk, io, workspace=64 * A + 128), INVALID)
    refused(mk, lambda: attn(mk, io, workspace=8 * A, size=4096), INVALID)
    refused(mk, lambda: mk._check("f", mk._lib_mk_kvq_attn_workspace(io, None)), INVALID)
    refused(mk, lambda: mk._check("f", mk._lib_mk_linear_workspace(linear_io(mk), None)), INVALID)
    assert mk.mk_kvq_attn_status(None) == INVALID and mk.mk_linear_status(None) == INVALID
    room = torch.zeros(1 << 16, dtype=torch.uint8)
    room = room[-room.data_ptr() % 256:]
    for call, i in ((mk.mk_kvq_attn, io), (mk.mk_linear, linear_io(mk))):
        for bad in (room[:1].expand(1 << 30), room[::2], room[:1 << 14].view(128, 128).t()):
            refused(mk, lambda: call(i, bad), INVALID)
        i.device = 1
        refused(mk, lambda: call(i, room), INVALID)


# ----------------------------------------------------------------- linear

def linear_io(mk, **over):
    f = dict(n_rows=4, n_in=256, n_out=384, dtype=0, act=0, x=A, x_stride=256, w=2 * A, w_stride=256, bias=3 * A,
             residual=4 * A, residual_stride=384, out=5 * A, out_stride=384)
    f.update(over)
    return mk.mk_linear_io(**f)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(n_rows=-1), INVALID), (dict(n_in=0), INVALID), (dict(n_out=0), INVALID),
    (dict(n_in=252), UNSUPPORTED), (dict(act=-1), INVALID), (dict(act=4), INVALID), (dict(x=0), INVALID),
    (dict(w=0), INVALID), (dict(out=0), INVALID), (dict(x=A + 8), INVALID), (dict(w=2 * A + 2), INVALID),
    (dict(x_stride=252), INVALID), (dict(x_stride=248), INVALID), (dict(w_stride=248), INVALID),
    (dict(w_stride=260), INVALID), (dict(out_stride=383), INVALID), (dict(residual_stride=383), INVALID),
    (dict(bias=3 * A + 1), INVALID), (dict(out=5 * A + 1), INVALID), (dict(out=A), INVALID), (dict(out=2 * A + 512), INVALID),
    (dict(out=3 * A), INVALID), (dict(out=4 * A, out_stride=400), INVALID), (dict(out=4 * A + 64), INVALID),
    (dict(n_rows=(1 << 31) - 1, n_out=(1 << 31) - 300, out_stride=1 << 32, residual=0), UNSUPPORTED)])
def test_linear_refusals(mk, over, status):
    refused(mk, lambda: mk._check("f", mk._lib_mk_linear(linear_io(mk, **over), 64 * A, 1 << 20, None)), status)


def test_linear_workspace_refusals(mk):
    for args in ((0, 1 << 20), (64 * A + 64, 1 << 20), (5 * A, 4096), (A, 4096), (64 * A, 128)):
        refused(mk, lambda: mk._check("f", mk._lib_mk_linear(linear_io(mk), *args, None)), INVALID)


def test_null_arguments(mk):
    for call in (lambda: mk._check("f", mk._lib_mk_qkv_append(None, None, None)),
                 lambda: mk._check("f", mk._lib_mk_kvq_read(None, None)),
                 lambda: mk._check("f", mk._lib_mk_kvq_attn(None, 64 * A, 1 << 30, None)),
                 lambda: mk._check("f", mk._lib_mk_kvq_attn_workspace(None, mk._i64())),
                 lambda: mk._check("f", mk._lib_mk_linear(None, 64 * A, 1 << 30, None)),
                 lambda: mk._check("f", mk._lib_mk_linear_workspace(None, mk._i64()))):
        refused(mk, call, INVALID)


# ---------------------------------------------------------------- binding

def test_binding_refuses_what_the_library_would_misread(mk):
    import torch
    u8 = torch.zeros(2, 2, 16, 8, dtype=torch.uint8)
    q = torch.zeros(2, 2, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int32)
    refused(mk, lambda: mk.make_kvq_cache(u8, u8[..., :1], u8, u8[..., :1]), INVALID)      # host memory
    refused(mk, lambda: mk.make_qkv_append_io(q, q, q, q, t, t.long()), INVALID)
    refused(mk, lambda: mk.make_linear_io(q[0], q[1], q[0]), INVALID)
    refused(mk, lambda: mk.make_kvq_attn_io(q, pools(mk, head_dim=16), q, t, t, t[None]), INVALID)
    refused(mk, lambda: mk.make_kvq_read_io(pools(mk), None, None, None), INVALID)
    # one thing at a time, with the device taken as given
    x = torch.zeros(6, 16, dtype=torch.bfloat16)
    assert mk._matrix("f", x[:, :8], 6, 8, x.dtype, -1) == (x.data_ptr(), 16)
    assert mk._matrix("f", x[:1, :8], 1, 8, x.dtype, -1) == (x.data_ptr(), 16)
    for bad, rows, cols in ((x.t(), 16, 6), (x, 6, 8), (x.half(), 6, 16), (x[:, ::2], 6, 8)):
        refused(mk, lambda: mk._matrix("f", bad, rows, cols, torch.bfloat16, -1), INVALID)
    kvq = pools(mk)
    kvq.device = 1
    refused(mk, lambda: mk._kvq_on("f", kvq, 0), INVALID)
    assert mk._kvq_on("f", kvq, 1) == bytes(kvq)


def test_packed_fields_are_the_structs(mk):
    """The packed layouts are those of the ctypes structs, field by field."""
    import struct
    four = mk.mk_kvq_cache.from_buffer_copy(struct.Struct("@4i6P").pack(*range(1, 11)))
    assert [getattr(four, f) for f, _ in four._fields_] == list(range(1, 11))
    for cls, pack in ((mk.mk_qkv_append_io, mk._pack_append), (mk.mk_kvq_read_io, mk._pack_read),
                      (mk.mk_kvq_attn_io, mk._pack_kvq_attn), (mk.mk_linear_io, mk._pack_linear)):
        values = [bytes(four) if f == "kvq" else i + 1 for i, (f, _) in enumerate(cls._fields_)]
        got = cls.from_buffer_copy(pack(*values))
        assert [bytes(getattr(got, f)) if f == "kvq" else getattr(got, f) for f, _ in cls._fields_] == values


@pytest.mark.parametrize("name", ["rows", "take_row", "convert", "issue_mmas"])
def test_warps_meet_before_instructions_for_whole_warps(name):
    assert sources.breaches(sources.body("kvq_wide.cu", name)) == []


@pytest.mark.parametrize("over,args,status", [
    ({}, (0, 1, 0, 0), INVALID), ({}, (2 * 10 ** 9 + 1, 1, 0, 0), INVALID), ({}, (10 ** 6, 5, 0, 0), INVALID),
    ({}, (10 ** 6, -1, 0, 0), INVALID), ({}, (10 ** 6, 1, -1, 0), INVALID), ({}, (10 ** 6, 1, 0, 2), INVALID),
    ({}, (10 ** 6, 2, 0, 1), INVALID), (dict(dtype=1), (10 ** 6, 1, 0, 0), UNSUPPORTED), (dict(w=0), (10 ** 6, 1, 0, 0), INVALID)])
def test_linear_waits_selftest_refusals(mk, over, args, status):
    assert mk._lib_mk_selftest_linear_waits(linear_io(mk, **over), 64 * A, 1 << 20, *args, None) == status
    assert mk._lib_mk_selftest_linear_waits(None, 64 * A, 1 << 20, 10 ** 6, 1, 0, 0, None) == INVALID


def test_linear_settles_what_was_given_up_behind_a_barrier():
    """The copies and products of work that was given up are waited for where every warp
    is through, by the word that all of them write, not by what one warp went through."""
    code = sources.body("linear.cu", "k_linear")
    meets = [m.start() for m in sources.re.finditer(r"\bmeet\(\)", code)]
    drains = [m.start() for m in sources.re.finditer(r"B\.drained|mbar_wait_bounded\(", code)]
    settled = code.index("gave_up =")
    assert len(meets) == 2 and meets[0] < settled < code.index("free_columns") and "B.abort" in code[settled:settled + 90]
    assert len(drains) > 2 and all(meets[0] < d < meets[1] for d in drains[1:])      # (the first is its initialisation)


@pytest.mark.parametrize("over,args,status", [
    ({}, (0, 1, 0), INVALID), ({}, (2 * 10 ** 9 + 1, 1, 0), INVALID), ({}, (10 ** 6, 10, 0), INVALID),
    ({}, (10 ** 6, -1, 0), INVALID), ({}, (10 ** 6, 1, -1), INVALID), (dict(dtype=1), (10 ** 6, 1, 0), UNSUPPORTED),
    ({}, (10 ** 6, 1, 0), UNSUPPORTED), (dict(n_rows=100, n_q_heads=7), (10 ** 6, 1, 0), INVALID),
    (dict(n_rows=100, lens=0), (10 ** 6, 1, 0), INVALID)])
def test_attention_waits_selftest_refusals(mk, over, args, status):
    kvq = pools(mk, head_dim=64)
    assert mk._lib_mk_selftest_kvq_waits(attn_io(mk, kvq, **over), 64 * A, 1 << 30, *args, None) == status
    assert mk._lib_mk_selftest_kvq_waits(attn_io(mk, n_rows=100), 64 * A, 1 << 30, 10 ** 6, 1, 0, None) == UNSUPPORTED
    assert mk._lib_mk_selftest_kvq_waits(None, 64 * A, 1 << 30, 10 ** 6, 1, 0, None) == INVALID


def test_attention_settles_what_was_given_up_behind_a_barrier():
    """As for the projection: the products are waited for where every warp is through, by
    the word that all of them write."""
    code = sources.body("kvq_wide.cu", "k_kvq_wide")
    last = code.rindex("__syncthreads()")
    tail = code[last:]
    assert code[:last].count("S.drained") == 1 and "mbar_wait_bounded" not in code[:last]      # its initialisation
    assert tail.index("S.abort") < tail.index("mma_commit(&S.drained)") < tail.index("mbar_wait_bounded(&S.drained") < tail.index("tmem_dealloc")


def test_linear_holds_tensor_memory_before_another_grid_may_come():
    """A dependent grid is let in behind the allocation, which waits without a limit, and
    no launch leaves room for a second CTA on an SM (the 227 KB that one can have)."""
    code = sources.body("linear.cu", "k_linear")
    assert code.count("pdl_launch_dependents(") == 1
    held = code[code.index("alloc_columns"):code.index("pdl_launch_dependents(")]
    assert ";" in held and "{" not in held                        # by the warp that took them, next
    text = open(sources.os.path.join(sources.CSRC, "linear.cu")).read()
    least = int(sources.re.search(r"kSmemLeast = (\d+) \* 1024;", text).group(1))
    assert 2 * (least + 1) > 227
    launch = text[text.index("mk_status launch("):]
    launch = launch[:launch.index("cudaLaunchKernelEx")]
    sets = sources.re.findall(r"\n  (?:if [^\n]*)?lc\.dynamicSmemBytes = [^;]*;", launch)
    assert "kSmemLeast" in sets[-1] and not sets[-1].startswith("\n  if")


def test_attention_holds_tensor_memory_before_another_grid_may_come():
    code = sources.body("kvq_wide.cu", "k_kvq_wide")
    assert code.count("pdl_launch_dependents(") == 1
    held = code[code.index("tmem_alloc"):code.index("pdl_launch_dependents(")]
    assert "tmem_relinquish" in held and "{" not in held


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("over", [
    dict(q_out=A + 2048, q_out_stride=1536), dict(q_out=A + 2560, q_out_stride=1536),        # over k, over v
    dict(q_out=A + 2048 - 2032, q_out_stride=1536, q=9 * A), dict(q_out=A + 2 * 1536 - 16, q_out_stride=1536, q=9 * A),
    dict(q_out=A - 2 * 1536 + 1040, q_out_stride=1536, q=9 * A), dict(q_out=A, q_out_stride=1024, q=9 * A),
    dict(n_rows=1, q_out=A + 1024, q=9 * A), dict(n_rows=1, q_out=A + 3056, q=9 * A)])
def test_append_refuses_q_out_over_k_and_v(mk, bits, over):
    refused(mk, lambda: mk.mk_qkv_append(None, append_io(mk, bits=bits, **over)), INVALID)


@pytest.mark.parametrize("over", [
    dict(v_cache=7 * A), dict(v_cache=7 * A + 16384), dict(k_cache=2 * A + 64), dict(v_cache=2 * A + 64), dict(k_cache=A),
    dict(v_cache=A), dict(k_cache=A + 3056, q=9 * A), dict(slots=7 * A + 8), dict(slots=8 * A + 8), dict(positions=7 * A + 4),
    dict(positions=8 * A + 32764), dict(q_norm=7 * A + 16), dict(k_norm=8 * A + 16), dict(v=7 * A, v_stride=256),
    dict(k=8 * A, k_stride=256), dict(n_slots=1 << 61), dict(n_slots=1 << 20)])
def test_append_refuses_what_overlaps_a_cache_in_16_bits(mk, over):
    r = mk.mk_rope_create(mk.make_rope_config(128))
    try:
        refused(mk, lambda: mk.mk_qkv_append(r, append_io(mk, bits=16, **over)), INVALID)
    finally:
        mk.mk_rope_destroy(r)


@pytest.mark.parametrize("over", [dict(k_exp=2 * A), dict(v_exp=2 * A + 64)])
def test_append_refuses_exponents_under_q_out(mk, over):
    refused(mk, lambda: mk.mk_qkv_append(None, append_io(mk, pools(mk, **over))), INVALID)


def test_a_single_row_has_no_stride(mk):
    """A view of one row of a tensor whose rows no call would take: nothing is between rows."""
    import torch
    x = torch.zeros(6, 60, dtype=torch.bfloat16)
    for one in (x[3:4, :16], x[3:4].expand(1, 60)[:, :16], x[3].as_strided((1, 16), (0, 1))):
        address, stride = mk._matrix("f", one, 1, 16, x.dtype, -1)
        assert address == one.data_ptr() and stride >= 16 and stride % 8 == 0
        address, stride = mk._rows("f", one.view(1, 2, 8), (1, 2, 8), x.dtype, -1)
        assert address == one.data_ptr() and stride >= 16 and stride % 8 == 0
    assert mk._matrix("f", x[:2, :16], 2, 16, x.dtype, -1)[1] == 60
    assert mk._rows("f", x[:2, :16].view(2, 2, 8), (2, 2, 8), x.dtype, -1)[1] == 60


def test_one_row_in_place_whatever_its_strides_say(mk):
    """Nothing to refuse (what follows is the GPU's absence or presence)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    for call in (lambda: mk._check("f", mk._lib_mk_linear(linear_io(mk, n_rows=1, out=4 * A, out_stride=400), 64 * A, 1 << 20, None)),
                 lambda: mk.mk_qkv_append(None, append_io(mk, n_rows=1, q_out=A))):
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.status not in (INVALID, UNSUPPORTED)


@pytest.mark.parametrize("eps", [float("nan"), -1.0, float("inf")])
def test_append_looks_at_eps_with_a_norm_only(mk, eps):
    empty = dict(n_rows=0, q=0, q_out=0, k=0, v=0, positions=0, slots=0, eps=eps)
    mk.mk_qkv_append(None, append_io(mk, **empty, q_norm=0, k_norm=0))
    for norms in (dict(q_norm=0), dict(k_norm=0), {}):
        refused(mk, lambda: mk.mk_qkv_append(None, append_io(mk, **empty, **norms)), INVALID)
