"""CPU tests of the paged-cache entry points: every refusal, before anything touches a GPU."""
import ctypes as C

import pytest
import torch

import lossless_depth_adaptive_gb300 as dexlib

EINVAL, ECAP = dexlib.DEX_EINVAL, dexlib.DEX_ECAPACITY


@pytest.fixture(scope="module", autouse=True)
def library():
    try:
        dexlib.lib()
    except dexlib.DexLibraryMissing:
        from lossless_depth_adaptive_gb300 import build
        build.build()


def kv(**over):
    # addresses are never followed: every call below is refused on the host
    f = dict(pages=1 << 20, table=1 << 21, page_stride=2 * 2 * 16 * 64, n_pages=8, page_size=16, n_kv_heads=2,
             head_dim=64, batch=3, table_width=4, table_stride=4, dtype=0)
    return dexlib.dex_paged_kv(**{**f, **over})


def append_args(**over):
    f = dict(q=1 << 22, k=1 << 23, v=1 << 24, q_out=1 << 25, q_stride=256, k_stride=128, v_stride=128, q_out_stride=256,
             seq=1 << 26, pos=1 << 26, n_tokens=5, n_heads=4, in_dtype=0, rope_theta=1e4)
    return dexlib.dex_append_args(**{**f, **over})


def attn_args(**over):
    f = dict(q=1 << 22, out=1 << 23, q_stride=256, out_stride=256, q_start=1 << 24, seq_len=1 << 24, n_tokens=5,
             n_heads=4, max_q=2, prefix_len=20, scale=0.125)
    return dexlib.dex_attention_args(**{**f, **over})


BAD_KV = [dict(head_dim=96), dict(head_dim=0), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(n_pages=0),
          dict(n_kv_heads=0), dict(n_kv_heads=-1), dict(n_kv_heads=2000), dict(batch=0), dict(batch=1025),
          dict(table_width=0), dict(table_stride=3), dict(dtype=2), dict(dtype=-1), dict(page_stride=4095),
          dict(page_stride=4100), dict(page_stride=-4096), dict(table_width=1 << 28, table_stride=1 << 28),
          dict(table_width=(1 << 27) - 31, table_stride=1 << 28)]


@pytest.mark.parametrize("bad", BAD_KV + [dict(pages=None), dict(table=None), dict(pages=(1 << 20) + 2)])
def test_bad_cache_is_refused(bad):
    L = dexlib.lib()
    assert L.dex_paged_append(C.byref(kv(**bad)), C.byref(append_args()), None, None) == EINVAL
    assert L.dex_prefix_attention(C.byref(kv(**bad)), C.byref(attn_args()), 1 << 20, 1 << 40, None, None) == EINVAL
    if bad in BAD_KV:
        n = C.c_size_t()
        assert L.dex_prefix_attention_workspace(C.byref(kv(**bad)), C.byref(attn_args()), C.byref(n)) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(q=None), dict(q_out=None), dict(n_tokens=-1),
    dict(n_heads=0), dict(k=(1 << 23) + 8), dict(v=(1 << 24) + 2), dict(q=(1 << 22) + 4), dict(q_out=(1 << 25) + 8),
    dict(k_stride=132), dict(v_stride=129), dict(q_stride=260), dict(q_out_stride=258), dict(q_out_stride=64),
    dict(in_dtype=1), dict(in_dtype=3), dict(in_dtype=-1), dict(rope_theta=0.5), dict(rope_theta=-1.0),
    dict(rope_theta=float("nan")), dict(rope_theta=float("inf")), dict(q=1 << 25, in_dtype=2), dict(q=1 << 25, q_stride=512),
    dict(n_tokens=(1 << 23) + 1), dict(n_tokens=2 ** 31 - 1)])
def test_bad_append_is_refused(bad):
    assert dexlib.lib().dex_paged_append(C.byref(kv()), C.byref(append_args(**bad)), None, None) == EINVAL


def test_null_structs_are_refused():
    L = dexlib.lib()
    n = C.c_size_t()
    assert L.dex_paged_append(None, C.byref(append_args()), None, None) == EINVAL
    assert L.dex_paged_append(C.byref(kv()), None, None, None) == EINVAL
    assert L.dex_prefix_attention(None, C.byref(attn_args()), 1 << 20, 1 << 40, None, None) == EINVAL
    assert L.dex_prefix_attention(C.byref(kv()), None, 1 << 20, 1 << 40, None, None) == EINVAL
    assert L.dex_prefix_attention_workspace(C.byref(kv()), None, C.byref(n)) == EINVAL
    assert L.dex_prefix_attention_workspace(C.byref(kv()), C.byref(attn_args()), None) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(n_tokens=-1), dict(n_tokens=1 << 24), dict(n_tokens=(1 << 23) + 1), dict(n_heads=0), dict(n_heads=5), dict(n_heads=258), dict(max_q=0),
    dict(max_q=-3), dict(prefix_len=-1), dict(prefix_len=65), dict(q=None), dict(out=None), dict(q_start=None),
    dict(seq_len=None), dict(q=(1 << 22) + 8), dict(out=(1 << 23) + 4), dict(q_stride=258), dict(out_stride=250),
    dict(out_stride=248), dict(scale=float("nan")), dict(scale=float("inf")), dict(tree_mask=1 << 20, max_q=65)])
def test_bad_attention_is_refused(bad):
    assert dexlib.lib().dex_prefix_attention(C.byref(kv()), C.byref(attn_args(**bad)), 1 << 20, 1 << 40, None,
                                             None) == EINVAL


@pytest.mark.parametrize("scale", [2.4e38, -3.0e38])
def test_scale_beyond_its_base_is_refused(scale):
    """Finite, but not in the base that the kernels use (times log2 e): it would make every score infinite."""
    assert dexlib.lib().dex_prefix_attention(C.byref(kv()), C.byref(attn_args(scale=scale)), 1 << 20, 1 << 40, None,
                                             None) == EINVAL


def test_workspace_size():
    """Given by sizes alone; too small or misaligned a workspace is refused."""
    L = dexlib.lib()
    c, a = kv(batch=64, n_kv_heads=8, page_stride=2 * 8 * 16 * 64), attn_args(n_tokens=64, n_heads=32, q_stride=2048, out_stride=2048)
    need = dexlib.dex_prefix_attention_workspace(c, a)
    assert need == dexlib.dex_prefix_attention_workspace(c, dexlib.dex_attention_args(
        n_tokens=64, n_heads=32, max_q=2, prefix_len=20))
    if need:
        assert L.dex_prefix_attention(C.byref(c), C.byref(a), 1 << 20, need - 1, None, None) == ECAP
        assert L.dex_prefix_attention(C.byref(c), C.byref(a), (1 << 20) + 16, need, None, None) == EINVAL
        assert L.dex_prefix_attention(C.byref(c), C.byref(a), None, need, None, None) == EINVAL


def test_largest_sizes():
    """The limits themselves are taken (their workspace can be told); one more is refused."""
    most = ((1 << 31) - 512) // 16
    c = kv(batch=1, table_width=most, table_stride=most, n_kv_heads=1)
    assert dexlib.dex_prefix_attention_workspace(c, attn_args(prefix_len=(1 << 31) - 512)) > 0
    c = kv(n_kv_heads=1)
    a = attn_args(n_tokens=1 << 23, n_heads=128, max_q=1 << 23, prefix_len=0)
    assert 0 < dexlib.dex_prefix_attention_workspace(c, a) < 1 << 40
    a.prefix_len, a.max_q, a.n_heads = 64, 1, 64   # a prefix of one tile is read by every sequence
    assert 0 < dexlib.dex_prefix_attention_workspace(c, a) < 1 << 40
    c = kv(n_kv_heads=1, table_width=2000, table_stride=2000)
    a.prefix_len = 32000   # shared: every row's result twice, in fp32
    assert dexlib.dex_prefix_attention_workspace(c, a) > (1 << 29) * 2 * 64 * 4
    a.n_tokens += 1
    assert dexlib.lib().dex_prefix_attention_workspace(C.byref(c), C.byref(a), C.byref(C.c_size_t())) == EINVAL


def test_cache_object_refuses_wrong_tensors():
    """The tensor checks of PagedCache come before the device check, so they show on the CPU."""
    def message(*args):
        with pytest.raises(dexlib.DexError) as e:
            dexlib.PagedCache(*args)
        assert e.value.code == EINVAL
        return str(e.value)

    pages = torch.zeros((4, 2, 2, 16, 64), dtype=torch.float16)
    table = torch.zeros((3, 4), dtype=torch.int32)
    assert "pages must be [" in message(pages[0], table)
    assert "bf16 or fp16" in message(pages.float(), table)
    assert "contiguous" in message(pages.transpose(3, 4), table)
    assert "table must" in message(pages, table.long())
    assert "table must" in message(pages, table[0])
    assert "table must" in message(pages, table.t())
    assert "workspace" in message(torch.zeros((4, 2, 2, 16, 32), dtype=torch.float16), table)   # head_dim 32
    assert "CUDA device" in message(pages, table)


def test_calls_refuse_wrong_tensors(monkeypatch):
    """append() and attention() on CPU tensors: shapes, types and strides first, then the device."""
    monkeypatch.setattr(dexlib.PagedCache, "_on_device", lambda self, **t: None)
    pages = torch.zeros((4, 2, 2, 16, 64), dtype=torch.float16)
    cache = dexlib.PagedCache(pages, torch.zeros((3, 4), dtype=torch.int32))
    monkeypatch.undo()
    k = torch.zeros((5, 2, 64), dtype=torch.float16)
    q = torch.zeros((5, 6, 64), dtype=torch.float16)
    idx = torch.zeros(5, dtype=torch.int32)
    start, lens = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def refused(fn, text):
        with pytest.raises(dexlib.DexError) as e:
            fn()
        assert e.value.code == EINVAL and text in str(e.value), str(e.value)

    refused(lambda: cache.append(k, k, idx, idx), "CUDA device")
    refused(lambda: cache.append(k.bfloat16(), k.bfloat16(), idx, idx), "type")
    refused(lambda: cache.append(k, k.float(), idx, idx), "type")
    refused(lambda: cache.append(k[:, :1], k, idx, idx), "k must be")
    refused(lambda: cache.append(k, k[:4], idx, idx), "v must be")
    refused(lambda: cache.append(k, k, idx[:4], idx), "seq")
    refused(lambda: cache.append(k, k, idx, idx.long()), "pos")
    refused(lambda: cache.append(k, k, idx, idx, rope_pos=idx[:2]), "rope_pos")
    refused(lambda: cache.append(k, k, idx, idx, q=q.transpose(0, 1)), "q must be")
    refused(lambda: cache.append(k, k, idx, idx, q=q.float()), "q must have")
    refused(lambda: cache.append(k, k, idx, idx, q=q, q_out=q.float()), "q_out must have")
    refused(lambda: cache.append(k, k, idx, idx, q_out=q), "q_out needs q")
    refused(lambda: cache.append(k, k, idx, idx, rejected=idx), "rejected")
    refused(lambda: cache.attention(q, start, lens, 1), "CUDA device")
    refused(lambda: cache.attention(q.float(), start, lens, 1), "type")
    refused(lambda: cache.attention(q, start[:3], lens, 1), "q_start")
    refused(lambda: cache.attention(q, start, lens.long(), 1), "seq_len")
    refused(lambda: cache.attention(q, start, lens, 0), "max_q")
    refused(lambda: cache.attention(q, start, lens, 2 ** 32 + 1), "max_q")
    refused(lambda: cache.attention(q, start, lens, 1, prefix_len=-1), "prefix_len")
    refused(lambda: cache.attention(q, start, lens, 1, prefix_len=40, prefix_table=idx[:2]), "prefix_table")
    refused(lambda: cache.attention(q, start, lens, 1, out=q[:, :3]), "out must be")
    refused(lambda: cache.attention(q, start, lens, 1, lse=torch.zeros((5, 5))), "lse")
    refused(lambda: cache.attention(q, start, lens, 1, tree_mask=idx), "tree_mask")
    refused(lambda: cache.attention(q, start, lens, 1, status=idx), "status")
