"""The history cache's entry points without a GPU: sizes, refusals before any
launch, and calls that have nothing to do."""
import ctypes

import pytest
import torch

import block_sparse_attention_kunlun_b200 as ba

FAKE = 1 << 20  # an aligned address that no refused call dereferences


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, page_table=FAKE, status=None, batch=3, max_pages=10,
             num_pages=20, page_size=64, kv_heads=2, head_dim=128)
    f.update(kw)
    return ba.BACache(*[f[name] for name, _ in ba.BACache._fields_])


def prob(batch=3, T=5, H=4, D=128, dt=ba.BA_BF16):
    return ba.BAProblem(batch, T, H, D, dt)


def write(c, dtype=ba.BA_BF16, k=FAKE, v=FAKE, offs=FAKE, starts=FAKE, rows=5):
    return ba.ba_cache_write(c, dtype, k, v, offs, starts, rows, stream=0)


def read(c, dtype=ba.BA_BF16, k=FAKE, v=FAKE, offs=FAKE, starts=FAKE, rows=5):
    return ba.ba_cache_read(c, dtype, offs, starts, rows, k, v, stream=0)


def summarize(c, starts=FAKE, ends=FAKE, out=FAKE):
    return ba.ba_cache_summarize(c, starts, ends, out, stream=0)


def select(c, p=None, q=FAKE, offs=FAKE, lens=FAKE, pos=None, summaries=FAKE, block=64, window=1, topk=4, mask=FAKE):
    return ba.ba_cache_select(c, p or prob(), q, offs, lens, pos, summaries, block, window, topk, mask, stream=0)


def fwd(c, p=None, q=FAKE, offs=FAKE, lens=FAKE, pos=None, tree=None, tree_words=0, mask=None, block=64, window=1,
        out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return ba.ba_cache_fwd(c, p or prob(), q, offs, lens, pos, tree, tree_words, mask, block, window, out, lse, ws,
                           workspace_bytes=ws_bytes, stream=0)


CALLS = [write, read, summarize, select, fwd]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k_scales=None), dict(v_scales=None), dict(page_table=None),
    dict(k=FAKE + 8), dict(v_scales=FAKE + 4), dict(page_table=FAKE + 2), dict(status=FAKE + 1),
    dict(batch=-1), dict(max_pages=0), dict(num_pages=0), dict(page_size=0), dict(kv_heads=0), dict(head_dim=0)])
def test_bad_caches_are_invalid(call, kw):
    assert call(cache(**kw)) == ba.BA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(head_dim=96),
                                dict(head_dim=32), dict(max_pages=1 << 25), dict(kv_heads=65536)])
def test_unsupported_caches(call, kw):
    assert call(cache(**kw)) == ba.BA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw", [dict(dtype=7), dict(rows=-1), dict(k=None), dict(v=None), dict(k=FAKE + 8),
                                dict(offs=None), dict(starts=None), dict(offs=FAKE + 2), dict(starts=FAKE + 1)])
def test_bad_rows(call, kw):
    assert call(cache(), **kw) == ba.BA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(starts=None), dict(ends=None), dict(out=None), dict(out=FAKE + 4),
                                dict(ends=FAKE + 3)])
def test_bad_summaries(kw):
    assert summarize(cache(), **kw) == ba.BA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [select, fwd])
@pytest.mark.parametrize("kw", [
    dict(p=prob(batch=2)), dict(p=prob(D=64)), dict(p=prob(H=3)), dict(p=prob(H=0)), dict(p=prob(T=-1)),
    dict(p=prob(dt=9)), dict(block=0), dict(window=0), dict(q=None), dict(q=FAKE + 8), dict(offs=None),
    dict(lens=None), dict(pos=FAKE + 2), dict(mask=FAKE + 2)])
def test_bad_queries(call, kw):
    assert call(cache(), **kw) == ba.BA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [select, fwd])
def test_unsupported_queries(call):
    assert call(cache(), p=prob(dt=ba.BA_F32)) == ba.BA_ERR_UNSUPPORTED
    assert call(cache(), p=prob(T=2 ** 30)) == ba.BA_ERR_UNSUPPORTED  # rows of a group: 2^31


def test_select_limits():
    assert select(cache(), topk=0) == ba.BA_ERR_INVALID_ARG
    assert select(cache(), summaries=None) == ba.BA_ERR_INVALID_ARG
    assert select(cache(), mask=None) == ba.BA_ERR_INVALID_ARG
    assert select(cache(max_pages=16385)) == ba.BA_ERR_UNSUPPORTED
    assert fwd(cache(max_pages=16385), mask=FAKE) == ba.BA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(tree=FAKE, tree_words=0), dict(tree_words=-1), dict(tree=FAKE + 2, tree_words=1),
                                dict(out=None), dict(lse=None), dict(out=FAKE + 2), dict(lse=FAKE + 2)])
def test_bad_attention_arguments(kw):
    assert fwd(cache(), **kw) == ba.BA_ERR_INVALID_ARG


def test_attention_workspace():
    c = cache(max_pages=4096)   # 262144 slots: few rows, so the slots are split
    need = ba.ba_cache_fwd_workspace_size(c, prob(), 1 << 20, 1)
    assert need > 0 and need % 256 == 0
    assert fwd(c, block=1 << 20, ws_bytes=need - 1) == ba.BA_ERR_INVALID_ARG
    assert fwd(c, block=1 << 20, ws=None) == ba.BA_ERR_INVALID_ARG
    assert fwd(c, block=1 << 20, ws=FAKE + 128) == ba.BA_ERR_INVALID_ARG
    # bad arguments size to 0
    assert ba.ba_cache_fwd_workspace_size(cache(page_size=8), prob(), 64, 1) == 0
    assert ba.ba_cache_fwd_workspace_size(c, prob(batch=2), 64, 1) == 0
    assert ba.ba_cache_fwd_workspace_size(c, prob(), 0, 1) == 0


@pytest.mark.parametrize("batch,T,heads,kv,pages", [(1, 1, 1, 1, 1), (256, 256, 8, 8, 64), (16, 16, 32, 8, 512),
                                                    (1, 2000, 8, 1, 4096), (1000, 1000, 64, 64, 16384)])
def test_attention_workspace_is_bounded(batch, T, heads, kv, pages):
    """The parts are float32 rows with two statistics: at most 16 to a query row and head beyond
    what fills the GPU."""
    c = cache(batch=batch, max_pages=pages, kv_heads=kv)
    for block, window in ((1, 1), (64, 1), (512, 4), (1 << 20, 1)):
        need = ba.ba_cache_fwd_workspace_size(c, prob(batch=batch, T=T, H=heads), block, window)
        row = 128 * 4 + 8
        assert need <= max(16 * T * heads, 1 << 16) * row + 1024


def test_nothing_to_do():
    assert write(cache(), rows=0, k=None, v=None) == ba.BA_OK
    assert read(cache(), rows=0, k=None, v=None) == ba.BA_OK
    assert summarize(cache(batch=0, page_table=None), starts=None, ends=None) == ba.BA_OK
    none = prob(T=0)
    assert select(cache(), p=none, q=None) == ba.BA_OK
    assert fwd(cache(), p=none, q=None, out=None) == ba.BA_OK


def test_null_structs():
    lib = ba._load()
    assert lib.ba_cache_write(None, 1, FAKE, FAKE, FAKE, FAKE, 1, None) == ba.BA_ERR_INVALID_ARG
    assert lib.ba_cache_fwd_workspace_size(ctypes.byref(cache()), None, 64, 1) == 0
    assert lib.ba_cache_fwd(ctypes.byref(cache()), None, FAKE, FAKE, FAKE, None, None, 0, None, 64, 1, FAKE, FAKE,
                            FAKE, 1 << 30, None) == ba.BA_ERR_INVALID_ARG


def test_the_binding_checks_its_tensors():
    t = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((4, 2, 16, 2), dtype=torch.uint8)
    table = torch.zeros((3, 5), dtype=torch.int32)
    for k, v, ks, vs, tb, what in (
            (t[0], t, s, s, table, "num_pages"), (t.float(), t, s, s, table, "k must"), (t, t[:2], s, s, table, "v must"),
            (t, t, s[..., :1], s, table, "k_scales"), (t, t, s, s, table.long(), "page_table"),
            (t, t, s, s, table[0], "page_table"), (t, t, s, s, table, "CUDA")):
        with pytest.raises(ValueError, match=what):
            ba.HistoryCache(k, v, ks, vs, tb, status=torch.zeros(1, dtype=torch.int32))
