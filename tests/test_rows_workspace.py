"""Workspace of the shared-prefix decode and the cross attention: sized by the
row heads that exist; refusals of the test-only stall (host side, no GPU needed)."""
import itertools

import pytest


@pytest.fixture(scope="module")
def Q():
    from bit_kv_cache_dqk_b200 import build
    build.build()
    from bit_kv_cache_dqk_b200 import dualqk
    return dualqk


def layer(Q, d=128, hq=32, hkv=8):
    return Q.layer_desc(d, hq, hkv, 256, 256, 256, 1 << 20)


MB = 1 << 20


@pytest.mark.parametrize("int2", [True, False])
def test_many_prefixes_of_few_sequences(Q, int2):
    size = Q.dqk_prefix_decode_workspace_size if int2 else Q.dqk_bf16_prefix_decode_workspace_size
    d = layer(Q)
    record = 528                                             # bytes of a record at head_dim 128
    for n, most in ((1, 2), (64, 60), (256, 64), (1024, 100)):
        got = size(d, n, n, 64, 64)
        # two records of every row head (group's and own) and, for each of 160 CTAs, those of an item that it shares
        least = (2 * 2 * n * 32 + 160 * 2 * min(128, 4 * n)) * record
        assert got <= least + 160 * 2 * 4 * record + n * 32 * 272 + 64 * 1024, (n, got, least)
        assert got <= most * MB, (n, got)
    assert size(d, 1, 1, 1, 0) < 200 * 1024


def test_small_cross_attention(Q):
    assert Q.dqk_bf16_cross_attention_workspace_size(layer(Q), 1, 1, 4) < 256 * 1024
    # many rows: no more than two segments a CTA
    assert Q.dqk_bf16_cross_attention_workspace_size(layer(Q), 4, 8192, 4096) <= 160 * 2 * 256 * 528 + 64 * 1024


@pytest.mark.parametrize("which", ["int2", "bf16", "cross"])
def test_grows_with_every_size(Q, which):
    """A workspace of the largest call serves every smaller one."""
    d = layer(Q, hq=16, hkv=4)
    batches, lists, pages, own = (1, 2, 9, 33, 200, 1500), (1, 2, 7, 64, 500), (1, 8, 9, 64, 4000), (0, 1, 9, 300)
    if which == "cross":
        def size(b, n, p, o):
            return Q.dqk_bf16_cross_attention_workspace_size(d, n, b, p)
        own = (0,)
    else:
        f = Q.dqk_prefix_decode_workspace_size if which == "int2" else Q.dqk_bf16_prefix_decode_workspace_size

        def size(b, n, p, o):
            return f(d, b, n, p, o)
    axes = (batches, lists, pages, own)
    got = {i: size(*(a[k] for a, k in zip(axes, i))) for i in itertools.product(*(range(len(a)) for a in axes))}
    for i, x in got.items():
        for axis in range(4):
            up = tuple(k + (axis == a) for a, k in enumerate(i))
            assert up not in got or got[up] >= x > 0, (i, up)


def test_stall_is_refused_as_the_plain_calls(Q):
    d = layer(Q)
    for bf16 in (0, 1):
        ok = [d, bf16, 256, Q.DQK_BF16, 4, 1, 256, 256, 256, 8, 256, 256, 2, 40, 256, Q.DQK_F32, None, 256, 64]
        assert Q.dqk_test_prefix_stall(*ok, stream=0, raise_on_error=False) == Q.DQK_ERR_WORKSPACE_TOO_SMALL
        bad = ok[:4] + [0] + ok[5:]
        assert Q.dqk_test_prefix_stall(*bad, stream=0, raise_on_error=False) == Q.DQK_ERR_INVALID_ARG
