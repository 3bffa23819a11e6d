"""Pins of the drafted-tree oracle: a path through a tree is single-query
decode after appending it, and verification leaves the target's distribution
unchanged. Host argument checks of the three calls run here too."""
import ctypes
import math

import numpy as np
import pytest

import synth
from oracle import attention, codecs, tree
from tests.helpers import entry_rows, lay_out, window_rows


def test_family_walks_to_the_root_and_stops_at_a_bad_parent():
    assert tree.family([-1, 0, 0, 1, 3], 4) == [4, 3, 1, 0]
    assert tree.family([-1, 0, 2], 2) == [2]      # its own parent
    assert tree.family([-1, -5, 1], 2) == [2, 1]


@pytest.mark.parametrize("cached,depth", [(0, 0), (5, 2), (126, 1), (127, 0), (131, 4), (300, 3)])
def test_a_path_equals_decode_after_appending_it(cached, depth):
    r = synth.rng(71)
    W, ratio, H = 128, 4, 3
    total = cached + depth + 1
    ents = entry_rows(r, -(-total // ratio), "fp8")
    rows = codecs.bf16_round(synth.normal(r, (total, 512)))
    main = lay_out([ents], 64, r, "fp8", max_blocks=4).seq(0)
    full = np.zeros((total, 512), dtype=np.uint16)
    full[:] = codecs.bf16_bits(rows)
    win = lay_out([(full, None)], 256, r, "bf16").seq(0)
    q = synth.normal(r, (H, 512)).astype(np.float64)
    ref = attention.decode_one(q, main, win, total, ratio, W, 1 / math.sqrt(512))
    parents = [-1] + list(range(depth))
    got, _ = tree.attend_node(q, depth, parents, rows[cached:].astype(np.float64), main, win, cached, ratio, W,
                              1 / math.sqrt(512))
    np.testing.assert_allclose(got, ref, rtol=0, atol=1e-12)


def test_window_rows_helper_is_what_the_tree_reads():
    r = synth.rng(72)
    vals, _ = window_rows(r, 10, 4)
    assert not vals[:6].any() and vals[6:].any()


@pytest.mark.parametrize("children,draft", [(1, True), (2, True), (3, True), (1, False), (2, False)])
def test_verification_leaves_the_target_distribution(children, draft):
    """Over all drafts (weighted by their probability) and random accept and
    sample numbers, the first new token has the target's distribution. 6000
    draws of a probability have a standard deviation of at most
    sqrt(1/4 / 6000) = 0.0065, and stratifying over the drafts lowers it."""
    p, q, draws = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.5, 0.3]), 6000
    parents = [-1] + [0] * children
    target, rows = np.stack([p] * (children + 1)), np.stack([q] * (children + 1))
    drafts = np.stack(np.meshgrid(*[np.arange(3)] * children, indexing="ij"), -1).reshape(-1, children)
    if not draft:
        drafts = np.arange(children)[None]
    got, r = np.zeros(3), synth.rng(5)
    for d in drafts:
        weight = (float(np.prod(q[d])) if draft else 1.0) / (draws // len(drafts))
        for _ in range(draws // len(drafts)):
            path, nxt = tree.verify(target, rows if draft else None, parents, [0] + list(d),
                                    r.random(children + 1), r.random())
            got[d[path[1] - 1] if len(path) > 1 else nxt] += weight
    assert np.abs(got - p).max() < 5 * 0.0065, got


def test_verify_edges():
    p = np.array([[0.0, 1.0, 0.0], [0.25, 0.25, 0.5]])
    # a guess with all the mass is accepted for every u < 1, one without never
    assert tree.verify(p, None, [-1, 0], [0, 1], [0.0, 0.999], 0.0) == ([0, 1], 0)
    assert tree.verify(p, None, [-1, 0], [0, 2], [0.0, 0.0], 0.3) == ([0], 1)
    # equal draft and target: accepted for every u < 1
    assert tree.verify(p, p, [-1, 0], [0, 1], [0.0, 0.999], 0.6)[0] == [0, 1]
    # nothing left after the refusals: drawn from the target's row
    assert tree.verify(p[:1], None, [-1], [0], [0.0], 0.9) == ([0], 1)
    # no mass at all
    assert tree.verify(np.zeros((1, 4)), None, [-1], [0], [0.0], 0.9) == ([0], -1)
    # the drawn token is the first whose sum exceeds u * total
    assert tree.verify(p[1:], None, [-1], [0], [0.0], 0.25) == ([0], 1)
    assert tree.verify(p[1:], None, [-1], [0], [0.0], 0.0) == ([0], 0)


# ------------------------------------------------------------------ host checks of the library's calls

FAKE = 0x10000


def _attend_status(**kw):
    from paged_compressed_kv_b200 import v4kv
    a = dict(q=FAKE, q_dtype=2, batch=1, heads=8, cu=FAKE, total=4, most=4, parents=FAKE, k_tree=FAKE, seq=FAKE,
             max_len=1024, ratio=4, window_len=128, topk=None, k=0, sm_scale=0.04, out=FAKE, ws=FAKE, rope=(1e6, 64, 448))
    main = v4kv._Paged(FAKE, FAKE, 4, 64, 512, 1, FAKE, 4)
    win = v4kv._Paged(FAKE, None, 4, 256, 512, 0, FAKE, 4)
    a.update(kw)
    main = a.get("main", main)
    return v4kv._lib.v4kv_tree_attention(
        a["q"], a["q_dtype"], a["batch"], a["heads"], a["cu"], a["total"], a["most"], a["parents"], a["k_tree"],
        ctypes.byref(main), ctypes.byref(win), a["seq"], a["max_len"], a["ratio"], a["window_len"], a["topk"],
        a["k"], a["sm_scale"], v4kv._Rope(*a["rope"]), a["out"], a["ws"], 1 << 30, None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), 1), (dict(cu=None), 1), (dict(total=-1), 1), (dict(most=0), 1), (dict(most=129), 1),
    (dict(window_len=3), 1), (dict(parents=None), 1), (dict(k_tree=None), 1), (dict(k_tree=FAKE + 8), 1),
    (dict(q=None), 1), (dict(q=FAKE + 4), 1), (dict(q_dtype=1), 1), (dict(heads=129), 2), (dict(heads=0), 2),
    (dict(ratio=8), 1), (dict(topk=FAKE, k=2049), 1), (dict(topk=FAKE, k=0), 1), (dict(sm_scale=-1.0), 1),
    (dict(sm_scale=float("nan")), 1), (dict(out=FAKE + 2), 1), (dict(rope=(1e6, 64, 480)), 1), (dict(seq=None), 1),
    (dict(max_len=-1), 1)])
def test_tree_attention_rejects(bad, status):
    assert _attend_status(**bad) == status


@pytest.mark.parametrize("sizes", [
    dict(total=1 << 28), dict(batch=1 << 24, window_len=1 << 10, max_len=1 << 20),
    dict(batch=64, heads=128, total=8192, most=128, max_len=(1 << 31) - 1),
    dict(batch=1 << 23, heads=128, total=1 << 23, most=128, max_len=0)])
def test_tree_attention_refuses_sizes_it_cannot_count(sizes):
    from paged_compressed_kv_b200 import v4kv
    assert _attend_status(**sizes) == v4kv.V4KV_ERR_UNSUPPORTED
    a = dict(batch=1, heads=8, total=4, most=4, max_len=1024, window_len=128)
    a.update(sizes)
    with pytest.raises(v4kv.V4KVError) as e:
        v4kv.v4kv_tree_workspace_size(a["batch"], a["heads"], a["total"], a["most"], a["max_len"], 4, a["window_len"],
                                      0, v4kv.V4KV_FP8_E4M3)
    assert e.value.status == v4kv.V4KV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(total=-1), dict(most=0), dict(most=129), dict(window_len=3), dict(max_len=-1), dict(k=2049),
    dict(k=-1), dict(ratio=8), dict(dtype=2), dict(dtype=9)])
def test_tree_workspace_size_rejects(bad):
    from paged_compressed_kv_b200 import v4kv
    a = dict(batch=1, heads=8, total=4, most=4, max_len=1024, ratio=4, window_len=128, k=0, dtype=v4kv.V4KV_FP8_E4M3)
    a.update(bad)
    with pytest.raises(v4kv.V4KVError) as e:
        v4kv.v4kv_tree_workspace_size(a["batch"], a["heads"], a["total"], a["most"], a["max_len"], a["ratio"],
                                      a["window_len"], a["k"], a["dtype"])
    assert e.value.status == v4kv.V4KV_ERR_INVALID_ARG


def test_verify_takes_values_that_are_not_positive_as_zero():
    nan = float("nan")
    target = [[0.5, 0.5, 0.0], [1.0, 0.0, 0.0]]
    # a draft's negative value or NaN at a token: accepted where the target has it, refused where not
    for bad in (-1.0, nan):
        assert tree.verify(target, [[0.5, bad, 0.5], [1, 0, 0]], [-1, 0], [0, 1], [0, 0.9], 0.0)[0] == [0, 1]
        assert tree.verify(target, [[0.5, 0.5, bad], [1, 0, 0]], [-1, 0], [0, 2], [0, 0.9], 0.0)[0] == [0]


def test_tree_attention_rejects_other_dims():
    from paged_compressed_kv_b200 import v4kv
    assert _attend_status(main=v4kv._Paged(FAKE, FAKE, 4, 64, 256, 1, FAKE, 4)) == 2
    assert _attend_status(main=v4kv._Paged(FAKE, None, 4, 64, 512, 1, FAKE, 4)) == 1


@pytest.mark.parametrize("bad", [
    dict(target=None), dict(target=FAKE + 8), dict(tdt=1), dict(draft=FAKE + 4), dict(draft=FAKE, ddt=1), dict(vocab=0),
    dict(stride=99), dict(batch=0), dict(cu=None), dict(total=-1), dict(most=0), dict(most=129), dict(parents=None),
    dict(tokens=None), dict(accept=None), dict(sample=None), dict(path=None), dict(n_path=None), dict(nxt=None)])
def test_tree_verify_rejects(bad):
    from paged_compressed_kv_b200 import v4kv
    a = dict(target=FAKE, tdt=2, draft=None, ddt=0, vocab=100, stride=100, batch=1, cu=FAKE, total=4, most=4,
             parents=FAKE, tokens=FAKE, accept=FAKE, sample=FAKE, path=FAKE, n_path=FAKE, nxt=FAKE)
    a.update(bad)
    assert v4kv._lib.v4kv_tree_verify(a["target"], a["tdt"], a["draft"], a["ddt"], a["vocab"], a["stride"], a["batch"],
                                      a["cu"], a["total"], a["most"], a["parents"], a["tokens"], a["accept"],
                                      a["sample"], a["path"], a["n_path"], a["nxt"], None, None) == 1


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=FAKE + 2), dict(gate=None), dict(gate=FAKE + 4), dict(dim=12), dict(dim=0), dict(dim=1032),
    dict(gate_dim=2), dict(batch=0), dict(cu=None), dict(total=-1), dict(most=0), dict(path=None), dict(n_path=None),
    dict(x_out=None), dict(gate_out=None), dict(capacity=-1), dict(cu_out=None)])
def test_tree_gather_rejects(bad):
    from paged_compressed_kv_b200 import v4kv
    a = dict(x=FAKE, gate=FAKE, dim=512, gate_dim=1, batch=1, cu=FAKE, total=4, most=4, path=FAKE, n_path=FAKE,
             x_out=FAKE, gate_out=FAKE, capacity=4, cu_out=FAKE)
    a.update(bad)
    assert v4kv._lib.v4kv_tree_gather(a["x"], a["gate"], a["dim"], a["gate_dim"], a["batch"], a["cu"], a["total"],
                                      a["most"], a["path"], a["n_path"], a["x_out"], a["gate_out"], a["capacity"],
                                      a["cu_out"], None, None) == 1


def test_binding_rejects_host_tensors_and_wrong_shapes():
    import torch

    from paged_compressed_kv_b200 import v4kv
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        v4kv.v4kv_tree_verify(torch.zeros(1, 8), i, i[:1], i[:1], torch.zeros(1), torch.zeros(1), 1,
                              torch.zeros(1, 1, dtype=torch.int32), i[:1], i[:1])
    with pytest.raises(ValueError):
        v4kv.v4kv_tree_gather(torch.zeros(1, 8, dtype=torch.bfloat16), torch.zeros(1), i, i[None, :1], i[:1],
                              torch.zeros(1, 8, dtype=torch.bfloat16), torch.zeros(1), i)
