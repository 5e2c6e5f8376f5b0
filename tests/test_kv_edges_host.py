"""CPU tests of the binding's refusals of arguments that the calls could not follow. Nothing is launched."""
import pytest
import torch

import segmented_gather_gemv_amd as sg


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_page_tables_whose_rows_share_memory_are_refused():
    """A row is read at its number times the row stride: of a table expanded over the batch, or of overlapping
    windows, that led past its memory."""
    start, lens = _i32(0, 1, 3), _i32(5, 6)
    table = torch.arange(8, dtype=torch.int32)
    for bad in (table[:4].expand(2, 4), table.as_strided((2, 4), (2, 1)), table[:1].expand(2, 1)):
        with pytest.raises(ValueError, match="page_table"):
            sg.sgmv_kv_batch(start, lens, bad, 3, 2, 6)
    wide = torch.zeros(3, 9, dtype=torch.int32)
    for good, ldp in ((table.view(2, 4), 4), (table.view(2, 4)[:, :3], 4), (wide[:2, 8:], 9), (wide[:2, :0], 9),
                      (table.as_strided((2, 1), (3, 1)), 3)):
        b = sg.sgmv_kv_batch(start, lens, good, 3, 2, 6)
        assert b.desc.ldp == ldp and b.desc.table_pages == good.shape[1]
        last = b.desc.ldp + good.shape[1] + good.storage_offset()  # of the entries up to row 1's end
        assert last <= good.untyped_storage().nbytes() // 4
    one = sg.sgmv_kv_batch(_i32(0, 3), _i32(5), table[:4].expand(1, 4), 3, 3, 6)  # the stride of one row says nothing
    assert one.desc.ldp == 4


def test_whole_numbers_past_32_bits_are_refused():
    """ctypes cuts them to 32 bits: 2^32 + 4 pages were 4, a window of 2^32 + 5 tokens was 5."""
    start, lens, table, big = _i32(0, 1, 3), _i32(5, 6), torch.zeros(2, 4, dtype=torch.int32), 2 ** 32
    for sizes in ((4 + big, 16, 2, 64), (4, 16 + big, 2, 64), (4, 16, 2 + big, 64), (4, 16, 2, 64 + big)):
        with pytest.raises(ValueError, match="32 bits"):
            sg.sgmv_kv_init(*sizes, torch.int8, "cpu")
    for sizes in ((3 + big, 2, 6), (3, 2 + big, 6), (3, 2, 6 + big), (3, 2, -big), (3, 2, 2 ** 31)):
        with pytest.raises(ValueError, match="32 bits"):
            sg.sgmv_kv_batch(start, lens, table, *sizes)
    c = sg.sgmv_kv_init(4, 16, 2, 64, torch.int8, "cpu")
    b = sg.sgmv_kv_batch(start, lens, table, 3, 2, 6)
    q = torch.zeros(3, 4, 64)
    for kw in (dict(window=big + 5), dict(n_split=big + 2), dict(window=-big)):
        with pytest.raises(ValueError, match="32 bits"):
            sg.sgmv_kv_attention(q, b, c, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            sg.sgmv_kv_attention_workspace(4, torch.float32, b, c, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        sg.sgmv_kv_attention_workspace(4 + big, torch.float32, b, c)
    with pytest.raises(ValueError, match="32 bits"):
        sg.sgmv_kv_read(b, c, start, big + 3)
    f, t = torch.zeros(3), torch.zeros(5, 10)
    with pytest.raises(ValueError, match="32 bits"):
        sg.sgmv_verify_drafts(t, None, _i32(0, 0, 0), start, f, f[:2], big + 2)


def test_launches_past_the_limit_of_work_items_are_refused():
    """A launch takes fewer than 2^32 work items. Nothing is launched here: pointers are not followed."""
    import ctypes

    from segmented_gather_gemv_amd import _serving as sv
    lib = sg.library()

    def need(T, heads, head_dim, n_split, max_q=4096, fmt=sg.KV_I8):
        c = sv._KvCache(0x10000, 0x20000, 0x30000, 0x40000, 4, 16, 2, head_dim, fmt)
        b = sv._KvBatch(0x50000, 0x60000, 0x70000, 4, 4, 2, T, max_q, 64)
        a = sv._Attention(0x80000, 0x90000, None, heads * head_dim, head_dim, heads * head_dim, head_dim, heads,
                          sg.SGMV_BF16, 0.125, 0, n_split)
        size = ctypes.c_size_t()
        return lib.sgmv_kv_attention_workspace(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c), ctypes.byref(size))

    # of the direct kernel, 8 of a row and head (256 of 32 of them); of the join, 64
    assert need(2 ** 24, 30, 112, 1) == sg.SGMV_OK
    assert need(2 ** 24, 32, 112, 1) == sg.SGMV_EUNSUPPORTED
    # of the tiled kernel, 2 of a row and head
    assert need(2 ** 24, 120, 128, 1) == sg.SGMV_OK
    assert need(2 ** 24, 120, 128, 2) == sg.SGMV_EUNSUPPORTED
    assert need(2 ** 21, 30, 128, 2) == sg.SGMV_OK
    assert need(2 ** 21, 32, 128, 2) == sg.SGMV_EUNSUPPORTED
