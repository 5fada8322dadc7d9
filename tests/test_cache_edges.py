"""Cached attention without a GPU: sizes at the edge of what the calls take."""

import precision_attention_video_b200 as pav


def params(**kw):
    base = dict(n_pages=10, page_size=16, H=32, Hkv=8, d=128, S=2, T=2000, max_pages=400, n_select=16)
    base.update(kw)
    return pav.make_cache_params(**base)


def test_workspace_has_no_logits_where_the_choice_refuses_the_sizes():
    # what sparse attention and append need is there; 2000 rows of 65536 pages
    # would have taken 33 GB of logits that no call can use
    lists = pav.cache_workspace_bytes(params(n_select=16, max_pages=16385))
    for kw in (dict(max_pages=65536), dict(max_pages=1 << 26), dict(max_pages=16384, H=8 * 129)):
        n = pav.cache_workspace_bytes(params(**kw))
        assert 0 < n < 1 << 29, kw
    assert lists < pav.cache_workspace_bytes(params(max_pages=16384))


def test_workspace_of_a_long_prompt_is_bounded():
    # logits for 4 GiB of rows at a time; beside them what grows with the rows
    # is some ten bytes a (row, head), and with the table the split means
    short, long = params(T=2000, max_pages=512), params(T=100000, max_pages=512)
    assert pav.cache_workspace_bytes(short) < 1 << 29
    assert pav.cache_workspace_bytes(long) < (1 << 32) + 100000 * (32 * 4 + 8 * 8 + 8) + (1 << 26)
    wide = params(T=4000, max_pages=16384)
    assert pav.cache_workspace_bytes(wide) < (1 << 32) + 2 * 8 * 16384 * 520 + (1 << 26)
    # a token a sequence: no split means
    assert pav.cache_workspace_bytes(params(T=3000, S=3000, max_pages=16384)) < (1 << 32) + (1 << 26)
