"""Host-side checks of the rotated appends, the shared-prefix decode and the
cross attention (no GPU needed): bad arguments are refused before anything
reaches a device."""
import pytest


@pytest.fixture(scope="module")
def Q():
    from bit_kv_cache_dqk_b200 import build
    build.build()
    from bit_kv_cache_dqk_b200 import dualqk
    return dualqk


A = 256   # an aligned address that is never touched


def layer(Q, **kw):
    a = dict(head_dim=128, num_q_heads=32, num_kv_heads=8, t_k=A, t_q=A, pool=A, num_pages=10)
    a.update(kw)
    return Q.layer_desc(**a)


def rope_status(Q, fn="dqk_rope_append", desc=None, rope=None, **kw):
    a = dict(k=A, k_stride=1024, v=A, v_stride=1024, q=A, q_stride=4096, q_out=A, q_out_stride=4096, dtype=Q.DQK_BF16,
             batch=1, new_lens=A, seq_lens_before=A, max_new=1, positions=None, page_table=A, max_pages=4)
    a.update(kw)
    desc = layer(Q) if desc is None else desc
    rope = Q.rope_desc(128, A, 100) if rope is None else rope
    return getattr(Q, fn)(desc, rope, stream=0, raise_on_error=False, **a)


@pytest.mark.parametrize("fn", ["dqk_rope_append", "dqk_bf16_rope_append"])
def test_rope_append_refusals(Q, fn):
    bad = lambda **kw: rope_status(Q, fn, **kw)  # noqa: E731
    for name in ("k", "v", "new_lens", "seq_lens_before", "page_table"):
        assert bad(**{name: None}) == Q.DQK_ERR_INVALID_ARG, name
    assert bad(q=None) == bad(q_out=None) == Q.DQK_ERR_INVALID_ARG          # one of the two
    for name in ("k", "v", "q", "q_out"):
        assert bad(**{name: A + 8}) == Q.DQK_ERR_INVALID_ARG, name          # not 16-byte aligned
    for name, least in (("k_stride", 1024), ("v_stride", 1024), ("q_stride", 4096), ("q_out_stride", 4096)):
        assert bad(**{name: least - 8}) == Q.DQK_ERR_INVALID_ARG, name      # rows overlap
        assert bad(**{name: least + 4}) == Q.DQK_ERR_INVALID_ARG, name      # rows not in 16-byte steps
    assert bad(q_out_stride=8192) == Q.DQK_ERR_INVALID_ARG                  # in place needs one stride
    assert bad(dtype=7) == bad(batch=0) == bad(max_pages=0) == bad(max_new=-1) == Q.DQK_ERR_INVALID_ARG
    assert bad(rope=Q.rope_desc(128, None, 100)) == bad(rope=Q.rope_desc(128, A + 4, 100)) == Q.DQK_ERR_INVALID_ARG
    assert bad(rope=Q.rope_desc(128, A, 0)) == bad(rope=Q.rope_desc(128, A, 100, interleaved=2)) == Q.DQK_ERR_INVALID_ARG
    for r in (0, 8, 120, 144, -16):
        assert bad(rope=Q.rope_desc(r, A, 100)) == Q.DQK_ERR_UNSUPPORTED, r
    assert bad(desc=layer(Q, head_dim=96)) == bad(desc=layer(Q, num_q_heads=24)) == Q.DQK_ERR_UNSUPPORTED
    assert bad(desc=layer(Q, pool=None)) == Q.DQK_ERR_INVALID_ARG
    assert bad(max_new=0) == Q.DQK_OK                                       # nothing to append
    if fn == "dqk_rope_append":
        assert bad(desc=layer(Q, t_k=A + 4)) == bad(desc=layer(Q, t_k=None)) == Q.DQK_ERR_INVALID_ARG


def prefix_status(Q, int2, desc=None, **kw):
    a = dict(q=A, q_dtype=Q.DQK_BF16, batch=4, n_prefixes=1, prefix_start=A, prefix_lens=A, prefix_table=A,
             max_prefix_pages=8, seq_lens=A, page_table=A, max_pages=2, sparsity_pct=40, out=A, out_dtype=Q.DQK_BF16,
             sel_out=None, workspace=A, workspace_bytes=1 << 40)
    a.update(kw)
    fn = Q.dqk_prefix_decode
    if not int2:
        a.pop("sparsity_pct")
        a.pop("sel_out")
        fn = Q.dqk_bf16_prefix_decode
    return fn(layer(Q) if desc is None else desc, stream=0, raise_on_error=False, **a)


@pytest.mark.parametrize("int2", [True, False])
def test_prefix_decode_refusals(Q, int2):
    bad = lambda **kw: prefix_status(Q, int2, **kw)  # noqa: E731
    for name in ("q", "prefix_start", "prefix_lens", "prefix_table", "seq_lens", "page_table", "out", "workspace"):
        assert bad(**{name: None}) == Q.DQK_ERR_INVALID_ARG, name
    for name, off in (("q", 8), ("out", 8), ("workspace", 128)):
        assert bad(**{name: A + off}) == Q.DQK_ERR_INVALID_ARG, name
    for name in ("batch", "n_prefixes", "max_prefix_pages"):
        assert bad(**{name: 0}) == Q.DQK_ERR_INVALID_ARG, name
    assert bad(max_pages=-1) == bad(q_dtype=5) == bad(out_dtype=5) == Q.DQK_ERR_INVALID_ARG
    assert bad(workspace_bytes=64) == Q.DQK_ERR_WORKSPACE_TOO_SMALL
    assert bad(max_prefix_pages=1 << 27) == bad(batch=1 << 27) == Q.DQK_ERR_UNSUPPORTED
    assert bad(desc=layer(Q, page_size=32)) == Q.DQK_ERR_UNSUPPORTED
    if int2:
        assert bad(sparsity_pct=100) == bad(desc=layer(Q, t_q=A + 4)) == bad(desc=layer(Q, t_q=None)) == Q.DQK_ERR_INVALID_ARG


def test_cross_attention_refusals(Q):
    def bad(desc=None, **kw):
        a = dict(q=A, q_dtype=Q.DQK_BF16, batch=2, total_q=5, q_start=A, kv_lens=A, page_table=A, max_pages=4, out=A,
                 out_dtype=Q.DQK_F32, workspace=A, workspace_bytes=1 << 40)
        a.update(kw)
        return Q.dqk_bf16_cross_attention(layer(Q) if desc is None else desc, stream=0, raise_on_error=False, **a)
    for name in ("q", "q_start", "kv_lens", "page_table", "out", "workspace"):
        assert bad(**{name: None}) == Q.DQK_ERR_INVALID_ARG, name
    for name in ("batch", "total_q", "max_pages"):
        assert bad(**{name: 0}) == Q.DQK_ERR_INVALID_ARG, name
    assert bad(workspace_bytes=64) == Q.DQK_ERR_WORKSPACE_TOO_SMALL
    assert bad(total_q=1 << 26) == Q.DQK_ERR_UNSUPPORTED
    assert bad(desc=layer(Q, head_dim=256)) == Q.DQK_ERR_UNSUPPORTED


def test_workspace_sizes(Q):
    """0 for what the calls refuse; growing with the batch."""
    d = layer(Q)
    assert Q.dqk_prefix_decode_workspace_size(d, 0, 1, 8, 2) == 0
    assert Q.dqk_prefix_decode_workspace_size(layer(Q, num_q_heads=24), 4, 1, 8, 2) == 0
    assert Q.dqk_bf16_prefix_decode_workspace_size(d, 4, 0, 8, 2) == 0
    assert Q.dqk_bf16_cross_attention_workspace_size(d, 4, 0, 8) == 0
    small, large = (Q.dqk_prefix_decode_workspace_size(d, b, 1, 64, 2) for b in (4, 400))
    assert 0 < small < large
    assert 0 < Q.dqk_bf16_prefix_decode_workspace_size(d, 4, 1, 64, 0) < Q.dqk_bf16_prefix_decode_workspace_size(d, 4, 1, 64, 2)
