"""Trees of drafted tokens on the GPU against the fp64 oracle: attention of
every node, verification with given random numbers, packing of accepted rows,
and one speculative step of all of them with the append."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import attention, codecs, tree
from oracle.rope import rope_rotate
from tests.helpers import entry_rows, lay_out, oracle_index, window_rows

pytestmark = pytest.mark.gpu

W = 128


def make_parents(r, n, shape):
    if shape == "chain":
        return [-1] + list(range(n - 1)) if n else []
    if shape == "star":
        return [-1] + [0] * (n - 1) if n else []
    if shape == "forest":  # every node a root
        return [-1] * n
    return [-1 if i == 0 else int(r.integers(max(0, (i - 1) // 4), i)) for i in range(n)]


class TreeCase:
    def __init__(self, seed, lens, counts, heads, ratio=4, main_dtype="fp8", win_dtype="bf16", shape="tree",
                 topk=0, window=W, spare=0, q_std=1.0):
        r = synth.rng(seed)
        self.lens, self.counts, self.H, self.ratio, self.W = list(lens), list(counts), heads, ratio, window
        spb = 256 // ratio
        ents = [entry_rows(r, -(-L // ratio), main_dtype) for L in lens]
        ents = [e if e[0].shape[0] else (np.zeros((0, 512), e[0].dtype), e[1]) for e in ents]
        self.main = lay_out(ents, spb, r, main_dtype,
                            max_blocks=max([-(-(-(-L // ratio)) // spb) for L in lens] + [1]))
        first = [max(0, L - window) // 256 for L in lens]
        self.win = lay_out([window_rows(r, L, window, win_dtype) for L in lens], 256, r, win_dtype, first_block=first,
                           max_blocks=max([-(-L // 256) for L in lens] + [1]))
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.N = int(self.cu[-1]) + spare
        self.parents = np.full(self.N, -1, dtype=np.int32)
        for b, n in enumerate(counts):
            self.parents[self.cu[b]:self.cu[b + 1]] = make_parents(r, n, shape)
        self.q = codecs.bf16_round(synth.normal(r, (self.N, heads, 512), q_std))
        self.k_tree = codecs.bf16_round(synth.normal(r, (self.N, 512)))
        self.topk = None
        if topk:
            self.topk = np.full((self.N, topk), -1, dtype=np.int32)
            for b, n in enumerate(counts):
                vis = max(0, lens[b] + 1 - window) // ratio
                for i in range(n):
                    m = min(topk, vis)
                    pick = np.sort(r.permutation(vis)[:m])
                    at = np.sort(r.permutation(topk)[:m])
                    self.topk[self.cu[b] + i, at] = pick
        self.max_nodes = max(max(counts), 1)
        self.max_len = max(lens)

    def device(self, q_fp32=False):
        d = {"main": self.main.to_cuda(), "win": self.win.to_cuda()}
        d["q"] = torch.from_numpy(self.q).cuda() if q_fp32 else synth.bf16_tensor(self.q).cuda()
        d["k_tree"] = synth.bf16_tensor(self.k_tree).cuda()
        d["cu"] = torch.from_numpy(self.cu).cuda()
        d["parents"] = torch.from_numpy(self.parents).cuda()
        d["lens"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        d["topk"] = torch.from_numpy(self.topk).cuda() if self.topk is not None else None
        d["out"] = torch.full((self.N, self.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        d["st"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        d["ws"] = self.workspace(d)
        return d

    def workspace(self, d):
        from paged_compressed_kv_b200 import v4kv
        n = v4kv.v4kv_tree_workspace_size(len(self.lens), self.H, self.N, self.max_nodes, self.max_len, self.ratio,
                                          self.W, 0 if self.topk is None else self.topk.shape[1], d["main"].dtype_code)
        # whatever an earlier call left there
        return torch.randint(0, 256, (max(n, 256),), dtype=torch.uint8, device="cuda")

    def run(self, d, stream=None, **kw):
        from paged_compressed_kv_b200 import v4kv
        v4kv.v4kv_tree_attention(d["q"], d["cu"], d["parents"], d["k_tree"], d["main"], d["win"], d["lens"],
                                 self.max_nodes, self.max_len, self.ratio, self.W, d["out"], d["ws"],
                                 topk=d["topk"], dev_status=d["st"], stream=stream, **kw)

    def oracle(self, b, i):
        lo = self.cu[b]
        return tree.attend_node(self.q[lo + i], i, self.parents[lo:self.cu[b + 1]], self.k_tree[lo:self.cu[b + 1]],
                                self.main.seq(b), self.win.seq(b), self.lens[b], self.ratio, self.W,
                                1 / math.sqrt(512), topk_row=None if self.topk is None else self.topk[lo + i])

    def check(self, out, nodes=None, q_fp32=False):
        """Every value against fp64. A weight carries at most 2^-9 from its two
        e4m3 terms (half a step of the second term of a value in [1, 2) is
        2^-9) and the result one bf16 rounding (2^-8). With bf16 queries the
        scores are sums of exact products; their fp32 accumulation, and that of
        the outputs, stays below 2^-12 at these sizes (512 products a score of
        magnitude below 8: 512 * 8 * 2^-24 / 2). An fp32 query adds 2^-9 of
        sum|q v| scale, below 2^-9 * 16 here (|q||v| / sqrt(512) at the drawn
        sizes), to each score, and twice that to a weight's ratio. A weight
        below 2^-21 of its block's largest may vanish: 2^-16 of the largest
        value covers any number of them here."""
        out = out.float().cpu().numpy().astype(np.float64)
        for b, n in enumerate(self.counts):
            for i in range(n) if nodes is None else [i for i in nodes if i < n]:
                ref, mass = self.oracle(b, i)
                got = out[self.cu[b] + i]
                tol = (2.0 ** -9 + 2.0 ** -11) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * np.abs(mass).max()
                if q_fp32:
                    tol += 2 * 2.0 ** -9 * 16 * mass
                bad = np.abs(got - ref) > tol
                assert not bad.any(), (b, i, np.abs(got - ref)[bad].max(), tol[bad].min(), int(bad.sum()))


def chosen(c, r, most=6):
    return sorted(set(int(x) for x in r.integers(0, c.max_nodes, most)) | {0, c.max_nodes - 1})


CASES = [
    # lens, counts, heads, extra
    ([1024], [5], 8, dict(main_dtype="bf16")),
    ([0], [1], 64, {}),
    ([0, 1, 2], [3, 0, 1], 64, dict(shape="forest")),
    ([127, 128, 129, 130, 131, 132], [2, 4, 1, 3, 2, 5], 16, {}),
    ([3000, 517, 640], [1, 128, 77], 1, dict(shape="chain")),
    ([2047], [64], 24, dict(shape="star")),
    ([5000, 90, 1300], [7, 2, 12], 64, {}),
    ([5000, 90, 1300], [7, 2, 12], 64, dict(win_dtype="fp8")),
    ([2600, 700], [5, 9], 128, dict(main_dtype="bf16", win_dtype="fp8", shape="chain")),
    ([70000, 300, 140], [3, 6, 2], 64, dict(ratio=128)),
    ([40000, 33000], [9, 4], 10, dict(ratio=128, main_dtype="bf16")),
    ([9000, 400, 100], [4, 6, 3], 64, dict(topk=300)),
    ([9000, 2000], [3, 2], 64, dict(topk=512, shape="chain")),
    ([3000, 150], [5, 2], 6, dict(topk=1)),
    ([3000, 2500], [2, 3], 100, dict(topk=2048, main_dtype="bf16")),
    ([1500, 800], [3, 40], 8, dict(window=300)),
    ([1500, 800], [3, 40], 8, dict(window=40)),
]


@pytest.mark.parametrize("lens,counts,heads,extra", CASES)
def test_attention_matches_the_oracle(lens, counts, heads, extra):
    c = TreeCase(801 + heads + lens[0], lens, counts, heads, spare=3, **extra)
    d = c.device()
    c.run(d)
    torch.cuda.synchronize()
    assert int(d["st"].item()) == 0
    c.check(d["out"], nodes=chosen(c, synth.rng(1)))
    assert (d["out"][c.cu[-1]:] == 7.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("heads,extra", [(64, {}), (8, dict(main_dtype="bf16")), (64, dict(topk=100))])
def test_attention_with_fp32_queries(heads, extra):
    c = TreeCase(840, [1800, 333], [6, 3], heads, **extra)
    d = c.device(q_fp32=True)
    c.run(d)
    c.check(d["out"], q_fp32=True)
    assert int(d["st"].item()) == 0


def two_terms(q, low=True):
    """q as the products take it: hi + lo / 16, e4m3 both, of the row scaled so that
    its largest magnitude is in [2^7, 2^8); the residual in half precision."""
    up = np.exp2(7.0 - np.floor(np.log2(np.abs(q).max(axis=-1, keepdims=True)))).astype(np.float32)
    x = (q * up).astype(np.float32)
    hi = codecs.e4m3_decode(codecs.e4m3_encode(x)).astype(np.float16)
    rest = ((x.astype(np.float16) - hi) * np.float16(16)).astype(np.float32)
    lo = codecs.e4m3_decode(codecs.e4m3_encode(rest))
    return (hi.astype(np.float64) + (lo / 16 if low else 0.0)) / up


@pytest.mark.parametrize("heads,extra", [(64, {}), (8, dict(main_dtype="bf16")), (64, dict(topk=100))])
def test_fp32_queries_are_held_in_two_terms(heads, extra):
    """With q rounded as the header says, an output is within the bound of bf16
    queries. The same bound does not hold for a q without its low terms."""
    c = TreeCase(842, [1800, 333], [6, 3], heads, **extra)
    c.q = synth.normal(synth.rng(843), c.q.shape)
    d = c.device(q_fp32=True)
    c.run(d)
    q = c.q
    c.q = two_terms(q)
    c.check(d["out"])
    c.q = two_terms(q, low=False)
    with pytest.raises(AssertionError):
        c.check(d["out"])
    assert int(d["st"].item()) == 0


def test_a_path_equals_decode_after_appending_it():
    """One chain per sequence: the last node's output against
    v4kv_decode_attention with the chain's rows written into the window. Each
    call is within its own bound of the same fp64 value; the decode's bound is
    1e-2 of the largest output, the tree's is smaller."""
    from paged_compressed_kv_b200 import v4kv
    c = TreeCase(850, [1021, 600, 128], [3, 3, 3], 64, shape="chain")
    d = c.device()
    c.run(d)
    win = c.win.to_cuda()
    for b, L in enumerate(c.lens):
        for i in range(3):
            page = int(c.win.bt[b, (L + i) // 256])
            assert page >= 0
            win.data[page, (L + i) % 256] = d["k_tree"][c.cu[b] + i]
    rows = [int(c.cu[b]) + 2 for b in range(3)]
    lens = d["lens"] + 3
    out = torch.empty(3, 64, 512, dtype=torch.bfloat16, device="cuda")
    n = v4kv.v4kv_workspace_size(v4kv.V4KV_OP_DECODE, 3, 64, 1024, 4, W, 0, d["main"].dtype_code)
    v4kv.v4kv_decode_attention(d["q"][rows].contiguous(), d["main"], win, lens, 1024, 4, W, out,
                               torch.empty(n, dtype=torch.uint8, device="cuda"), dev_status=d["st"])
    a, b = d["out"][rows].float(), out.float()
    assert float((a - b).abs().max()) <= 2e-2 * float(b.abs().max())
    assert int(d["st"].item()) == 0


@pytest.mark.parametrize("main_dtype,win_dtype", [("fp8", "bf16"), ("fp8", "fp8"), ("bf16", "bf16")])
def test_rows_that_are_not_attended_may_hold_anything(main_dtype, win_dtype):
    """NaN and infinities in sibling nodes, in slots behind the visible entries,
    before the window and behind the cached tokens change nothing."""
    c = TreeCase(860, [1100, 523], [9, 6], 64, main_dtype=main_dtype, win_dtype=win_dtype)
    clean, dirty = c.device(), c.device()
    c.run(clean)
    bad16 = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(torch.bfloat16)
    for b, L in enumerate(c.lens):
        vis = max(0, L + max(c.counts) - W) // 4
        for j in range(vis, -(-L // 4)):
            page = int(c.main.bt[b, j // 64])
            if main_dtype == "fp8":
                dirty["main"].data[page, j % 64] = 0x7F if j % 2 else 0xFF
                dirty["main"].scales[page, j % 64] = float("nan") if j % 3 else float("inf")
            else:
                dirty["main"].data[page, j % 64] = bad16[j % 3]
        for t in list(range(max(0, L - W) // 256 * 256, max(0, L + 1 - W))) + list(range(L, -(-L // 256) * 256)):
            page = int(c.win.bt[b, t // 256])
            if win_dtype == "fp8":
                dirty["win"].data[page, t % 256] = 0x7F
                dirty["win"].scales[page, t % 256] = float("nan")
            else:
                dirty["win"].data[page, t % 256] = bad16[t % 3]
    c.run(dirty)
    assert torch.equal(clean["out"], dirty["out"])
    # a node's row reaches its own descendants only
    hit = 3
    dirty["k_tree"][int(c.cu[0]) + hit] = bad16[0]
    dirty["k_tree"][int(c.cu[1]) + hit, 17] = float("inf")
    c.run(dirty)
    for b in range(2):
        for i in range(c.counts[b]):
            row = int(c.cu[b]) + i
            if hit in tree.family(c.parents[c.cu[b]:c.cu[b + 1]], i):
                # the formula gives NaN at the dims that hold it; elsewhere too where the score is not -inf
                assert torch.isnan(dirty["out"][row] if b == 0 else dirty["out"][row, :, 17]).all()
            else:
                assert torch.equal(dirty["out"][row], clean["out"][row])


@pytest.mark.parametrize("heads,q_fp32", [(64, False), (10, True)])
def test_a_query_that_is_not_finite_reaches_its_own_row_only(heads, q_fp32):
    c = TreeCase(864, [1500, 400], [4, 3], heads)
    d = c.device(q_fp32=q_fp32)
    c.run(d)
    clean = d["out"].clone()
    bad = [(1, 3, 100, float("nan")), (2, 0, 0, float("inf")), (6, heads - 1, 511, -float("inf"))]
    for node, head, dim, value in bad:
        d["q"][node, head, dim] = value
    c.run(d)
    for node, head, _, _ in bad:
        assert torch.isnan(d["out"][node, head]).all()
        d["out"][node, head] = clean[node, head]
    assert torch.equal(d["out"], clean)


def test_entries_visible_to_the_deeper_nodes_only():
    """Entries that only the deeper nodes of a chain see hold NaN codes."""
    c = TreeCase(861, [1027], [14], 64, shape="chain")
    d = c.device()
    c.run(d)
    clean = d["out"].clone()
    L = 1027
    j = (L + 1 - W) // 4 + 1  # visible from depth 4 * (j + 1) - (L + 1 - W) on
    first = 4 * (j + 1) - (L + 1 - W)
    assert 0 < first < 13
    d["main"].data[int(c.main.bt[0, j // 64]), j % 64, 5] = 0x7F
    c.run(d)
    assert torch.equal(d["out"][:first], clean[:first])
    assert torch.isnan(d["out"][first:]).all()


def test_scales_of_any_value():
    c = TreeCase(862, [1500], [4], 64)
    r = synth.rng(9)
    c.main.scales[:] *= np.exp2(r.integers(-12, 4, c.main.scales.shape)).astype(np.float32)
    c.main.scales[r.random(c.main.scales.shape) < 0.1] = 0.0
    c.main.scales[r.random(c.main.scales.shape) < 0.2] *= -1.0
    d = c.device()
    c.run(d)
    c.check(d["out"])


def check_finite(c, d, nodes=None):
    """TreeCase.check lets a NaN pass: it is not above a tolerance."""
    assert torch.isfinite(d["out"][:int(c.cu[-1])].float()).all()
    c.check(d["out"], nodes=nodes)


@pytest.mark.parametrize("lens,counts,heads,extra", CASES)
def test_outputs_of_ordinary_calls_are_finite(lens, counts, heads, extra):
    c = TreeCase(802 + heads + lens[0], lens, counts, heads, **extra)
    d = c.device()
    c.run(d)
    assert torch.isfinite(d["out"][:int(c.cu[-1])].float()).all()


def scored(c, log2_score):
    """Queries that give each node's own row this score."""
    k = c.k_tree[:, None].astype(np.float64)
    c.q = codecs.bf16_round(np.broadcast_to(k * (log2_score * math.log(2) * math.sqrt(512)) /
                                            (k * k).sum(-1, keepdims=True), c.q.shape).astype(np.float32))


@pytest.mark.parametrize("log2_score", [2, 7])
@pytest.mark.parametrize("heads", [64, 6])
def test_a_window_of_zeros_beside_a_drafted_token(heads, log2_score):
    c = TreeCase(1000 + heads, [127, 40], [1, 3], heads)
    c.win.data[:] = 0
    c.k_tree = codecs.bf16_round(c.k_tree * 3)
    scored(c, log2_score)
    d = c.device()
    c.run(d)
    check_finite(c, d)


def test_a_drafted_token_of_zeros_alone_in_its_block():
    """96 ordinary tokens, then the node: its 32 items are its own row alone."""
    c = TreeCase(1003, [96, 128, 31], [1, 2, 4], 64)
    c.k_tree[[0, 2, 3]] = 0
    d = c.device()
    c.run(d)
    check_finite(c, d)


@pytest.mark.parametrize("lens,counts,extra", [
    ([3000], [3], {}), ([3000, 900], [8, 8], {}), ([2600, 700], [3, 5], dict(topk=200)),
    ([3000], [3], dict(main_dtype="fp8"))])
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0, 2.0 ** 6])
def test_rows_of_zeros_beside_others(lens, counts, extra, size):
    """Runs of zero rows of every kind, and single ones, beside small, ordinary
    and large rows (scores stay below 8)."""
    c = TreeCase(1010 + len(lens), lens, counts, 64, **dict(dict(main_dtype="bf16"), **extra))
    r = synth.rng(11)
    c.q = codecs.bf16_round(c.q * np.float32(1.0 / size))
    c.k_tree = codecs.bf16_round(c.k_tree * np.float32(size))
    c.win.data[:] = codecs.bf16_bits(codecs.bf16_to_f32(c.win.data) * np.float32(size))
    if c.main.dtype == "bf16":
        c.main.data[:] = codecs.bf16_bits(codecs.bf16_to_f32(c.main.data) * np.float32(size))
        gone = c.main.data
    else:
        c.main.scales *= np.float32(size)
        gone = c.main.scales
    gone[1] = 0
    gone[r.random(c.main.data.shape[:2]) < 0.2] = 0
    c.win.data[r.random(c.win.data.shape[:2]) < 0.2] = 0
    c.win.data[:, 40:120] = 0
    c.k_tree[1::3] = 0
    d = c.device()
    c.run(d)
    check_finite(c, d, nodes=chosen(c, synth.rng(2)))
    assert int(d["st"].item()) == 0


@pytest.mark.parametrize("lens,counts,extra", [
    ([3000], [3], {}), ([3000, 900], [8, 8], dict(win_dtype="fp8")), ([2600, 700], [3, 5], dict(topk=200)),
    ([900, 500], [3, 7], dict(heads=6)), ([40000, 33000], [8, 3], dict(ratio=128)), ([40000], [2], dict(ratio=128))])
@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** -12, 1.0])
def test_fp8_rows_of_zero_codes(lens, counts, extra, size):
    """Rows of zeros as the compressor writes them, codes 0 and the scale 1, beside
    small and ordinary rows whose scales are far below it."""
    c = TreeCase(1060 + len(lens), lens, counts, **dict(dict(heads=64), **extra))
    r = synth.rng(16)
    c.q = codecs.bf16_round(c.q * np.float32(1.0 / size))
    c.k_tree = codecs.bf16_round(c.k_tree * np.float32(size))
    for pool in (c.main, c.win):
        if pool.dtype == "bf16":
            pool.data[:] = codecs.bf16_bits(codecs.bf16_to_f32(pool.data) * np.float32(size))
            continue
        pool.scales *= np.float32(size)
        gone = r.random(pool.scales.shape) < 0.2
        gone[0] = True
        gone[r.random(gone.shape) < 0.02] = True
        pool.data[gone] = np.where(r.random((int(gone.sum()), 512)) < 0.5, 0x80, 0)  # either zero
        pool.scales[gone] = 1.0
    d = c.device()
    c.run(d)
    check_finite(c, d, nodes=chosen(c, synth.rng(2)))
    assert int(d["st"].item()) == 0


def test_nothing_but_zeros():
    """An output of zeros, split over the blocks or not."""
    c = TreeCase(1020, [9000, 90], [2, 3], 64, main_dtype="bf16")
    c.main.data[:], c.win.data[:], c.k_tree[:] = 0, 0, 0
    d = c.device()
    c.run(d)
    assert not d["out"].any()


@pytest.mark.parametrize("heads", [64, 8])
def test_zeros_in_a_long_context_that_blocks_share(heads):
    """Partial results with and without zero rows are joined."""
    c = TreeCase(1021, [40001], [3], heads, main_dtype="bf16")
    c.main.data[synth.rng(12).random(c.main.data.shape[0]) < 0.3] = 0
    d = c.device()
    c.run(d)
    check_finite(c, d)


def check_small(c, d):
    """As TreeCase.check, with half a step of bf16's subnormal values, and with what rows
    may hold that count as zeros: a scale below 2^-76 or 2^-60 of the largest. A bf16 row of
    largest magnitude A has the scale 2^(floor(log2 A) - 7), so either kind's values are
    below 2^9 scales."""
    scales = [np.abs(p.scales.astype(np.float64)).ravel() if p.dtype == "fp8" else
              np.abs(codecs.bf16_to_f32(p.data).astype(np.float64)).max(axis=-1).ravel() for p in (c.main, c.win)]
    scales.append(np.abs(c.k_tree.astype(np.float64)).max(axis=-1))
    for k, of_rows in enumerate((c.main.dtype == "bf16", c.win.dtype == "bf16", True)):
        if of_rows:
            _, e = np.frexp(scales[k])
            scales[k] = np.where(scales[k] > 0, np.ldexp(1.0, e - 8), 0.0)
    scales = np.concatenate(scales)
    gone = scales[scales < max(2.0 ** -76, 2.0 ** -60 * scales.max())]
    lost = 2.0 ** 9 * gone.max() if gone.size else 0.0
    out = d["out"].float().cpu().numpy().astype(np.float64)
    for b, n in enumerate(c.counts):
        for i in range(n):
            ref, mass = c.oracle(b, i)
            tol = (2.0 ** -9 + 2.0 ** -11) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mass.max() + 2.0 ** -133 + lost
            fine = np.abs(out[c.cu[b] + i] - ref) <= tol
            assert fine.all(), (b, i, int((~fine).sum()))


@pytest.mark.parametrize("power", [-149, -135, -127, -120, -100, -77, -76, -65, -50, -20])
@pytest.mark.parametrize("lens,counts,extra", [([1500], [4], {}), ([40001], [2], dict(heads=8)),
                                               ([2600, 700], [3, 5], dict(topk=200))])
def test_fp8_scales_near_zero(lens, counts, extra, power):
    """Entries that count in the normaliser and hardly or not in the value: all of them,
    some of them, of either sign, down to the smallest fp32 number."""
    c = TreeCase(1030, lens, counts, **dict(dict(heads=64), **extra))
    r = synth.rng(13)
    tiny = np.float32(2.0) ** power if power > -127 else np.ldexp(np.float32(1), power)
    keep = c.main.scales.copy()
    for some in (1.1, 0.5):
        c.main.scales[:] = np.where(r.random(keep.shape) < some, tiny, keep)
        c.main.scales[r.random(keep.shape) < 0.2] *= -1.0
        d = c.device()
        c.run(d)
        check_small(c, d)


def test_fp8_scales_of_all_sizes_at_once():
    c = TreeCase(1031, [3000, 400], [5, 3], 64, win_dtype="fp8")
    r = synth.rng(14)
    for pool in (c.main, c.win):
        powers = r.choice([-149, -140, -128, -126, -110, -80, -70, -45, -20, 0], pool.scales.shape)
        pool.scales[:] = np.where(powers < 0, np.ldexp(np.float32(1), powers), pool.scales)
        pool.scales[r.random(pool.scales.shape) < 0.1] = 0.0
    d = c.device()
    c.run(d)
    check_small(c, d)


@pytest.mark.parametrize("power", [-130, -118, -100, -68, -60, -36, 36, 60, 100])
@pytest.mark.parametrize("main_dtype", ["bf16", "fp8"])
def test_rows_of_any_magnitude(main_dtype, power):
    """All rows near 2^power, with queries that keep the scores ordinary where
    that is possible; then beside ordinary rows."""
    c = TreeCase(1040, [1500, 300], [4, 3], 64, main_dtype=main_dtype)
    size = np.ldexp(np.float64(1), power)

    def sized(x):
        return codecs.bf16_round((x.astype(np.float64) * size).astype(np.float32))

    r = synth.rng(15)
    q, win, main = c.q.copy(), c.win.data.copy(), c.main.data.copy()
    scales = None if c.main.scales is None else c.main.scales.copy()
    c.k_tree = sized(c.k_tree)
    c.q = codecs.bf16_round((q / max(size, 2.0 ** -100)).astype(np.float32))
    for some in (1.1, 0.5):
        if some < 1:
            c.q = codecs.bf16_round((q / max(size, 1.0)).astype(np.float32))
        at = r.random(win.shape[:2])[..., None] < some
        c.win.data[:] = np.where(at, codecs.bf16_bits(sized(codecs.bf16_to_f32(win))), win)
        at = r.random(main.shape[:2]) < some
        if scales is None:
            c.main.data[:] = np.where(at[..., None], codecs.bf16_bits(sized(codecs.bf16_to_f32(main))), main)
        else:
            c.main.scales[:] = np.where(at, (scales.astype(np.float64) * size).astype(np.float32), scales)
        d = c.device()
        c.run(d)
        check_small(c, d)
        assert int(d["st"].item()) == 0


def test_own_entries_chosen_by_the_indexer():
    """v4kv_index_topk with a node per row, then the nodes' attention over what it chose."""
    from paged_compressed_kv_b200 import v4kv
    k = 48
    c = TreeCase(1050, [900, 120, 133], [5, 2, 6], 64, topk=k)
    r = synth.rng(1051)
    keys = lay_out([codecs.quantize_entry(synth.normal(r, (-(-L // 4), 128))) for L in c.lens], 64, r, "fp8")
    q_idx = synth.normal(r, (c.N, 128))
    seq = np.repeat(np.arange(3), c.counts)
    depth = [len(tree.family(c.parents[c.cu[b]:c.cu[b + 1]], n - c.cu[b])) - 1 for n, b in enumerate(seq)]
    ends = [c.lens[b] + depth[n] + 1 for n, b in enumerate(seq)]
    d = c.device()
    pool = keys.to_cuda()
    pool.block_table = pool.block_table[torch.from_numpy(seq).cuda()].contiguous()
    n = v4kv.v4kv_workspace_size(v4kv.V4KV_OP_INDEX_TOPK, c.N, 1, max(ends), 4, W, k, v4kv.V4KV_FP8_E4M3, 128)
    v4kv.v4kv_index_topk(torch.from_numpy(q_idx).cuda(), pool, torch.tensor(ends, dtype=torch.int32, device="cuda"),
                         max(ends), 4, W, k, d["topk"], torch.empty(max(n, 256), dtype=torch.uint8, device="cuda"),
                         dev_status=d["st"])
    c.run(d)
    assert int(d["st"].item()) == 0
    c.topk = d["topk"].cpu().numpy()
    for n, b in enumerate(seq):
        assert np.array_equal(c.topk[n], oracle_index(q_idx[n], keys, b, ends[n], 4, W, k)[0])
    assert (c.topk[5] >= 0).sum() < (c.topk[12] >= 0).sum() < k
    c.check(d["out"])


def test_scores_that_grow_along_the_context():
    """A query along one direction whose entries' magnitude grows: the running
    maximum rises again and again, by far more than any fixed range."""
    c = TreeCase(863, [3000], [3], 64)
    direction = np.sign(c.q[:, :1].mean(axis=(0, 1)))[None, None]
    c.q = codecs.bf16_round(np.broadcast_to(direction, c.q.shape) * (1 + 0.01 * c.q))
    flat = codecs.e4m3_decode(c.main.data) * c.main.scales[..., None]
    for j in range(-(-3000 // 4)):
        page = int(c.main.bt[0, j // 64])
        flat[page, j % 64] = 0.02 * flat[page, j % 64] + direction[0, 0] * 0.01 * j
    codes, scales = codecs.quantize_entry(flat.reshape(-1, 512).astype(np.float32))
    c.main.data[:] = codes.reshape(c.main.data.shape)
    c.main.scales[:] = scales.reshape(c.main.scales.shape)
    d = c.device()
    c.run(d)
    out = d["out"].float().cpu().numpy()
    for i in range(3):
        ref, mass = c.oracle(0, i)
        # scores reach 170 here: their fp32 sums are off by up to 512 * 170 * 2^-24
        tol = (2.0 ** -9 + 2 * 512 * 170 * 2.0 ** -24) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mass.max()
        assert (np.abs(out[i] - ref) <= tol).all()


def test_references_that_rise_in_every_tile():
    """Scores that pass the running reference in each of twelve tiles: O, sums and
    scales are raised between the products, with the same bits in every run."""
    c = TreeCase(866, [6000], [9], 64)
    direction = np.sign(c.q[:, :1].mean(axis=(0, 1)))
    c.q = codecs.bf16_round(np.broadcast_to(direction[None, None], c.q.shape) * (1 + 0.01 * c.q))
    flat = codecs.e4m3_decode(c.main.data) * c.main.scales[..., None]
    for j in range(1500):
        page = int(c.main.bt[0, j // 64])
        flat[page, j % 64] = 0.02 * flat[page, j % 64] + direction * 0.02 * j
    codes, scales = codecs.quantize_entry(flat.reshape(-1, 512).astype(np.float32))
    c.main.data[:] = codes.reshape(c.main.data.shape)
    c.main.scales[:] = scales.reshape(c.main.scales.shape)
    d = c.device()
    c.run(d)
    first = d["out"].clone()
    out = first.float().cpu().numpy()
    for i in (0, 4, 8):
        ref, mass = c.oracle(0, i)
        # scores reach 680 here: their fp32 sums are off by up to 512 * 680 * 2^-24
        tol = (2.0 ** -9 + 2 * 512 * 680 * 2.0 ** -24) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mass.max()
        assert (np.abs(out[i] - ref) <= tol).all()
    for _ in range(30):
        d["out"].fill_(7.0)
        c.run(d)
        assert torch.equal(d["out"], first)


def test_bad_inputs_are_flagged_and_skipped():
    from paged_compressed_kv_b200 import v4kv
    c = TreeCase(870, [900, 700], [5, 4], 64)
    d = c.device()
    c.run(d)
    clean = d["out"].clone()
    # a parent behind its child: the child is a root
    d["parents"][2] = 2
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_BAD_INDEX
    keep = c.parents.copy()
    c.parents[2] = -1
    c.check(d["out"])
    c.parents = keep
    # a page outside the pool: its entries are left out
    d = c.device()
    d["main"].block_table[1, 0] = 10 ** 6
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_BAD_PAGE
    assert torch.equal(d["out"][:5], clean[:5])
    # a length above the host's bound is clamped, a sequence with too many nodes cut
    d = c.device()
    d["lens"][0] = 10 ** 6
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_OVERFLOW
    assert torch.equal(d["out"][:5], clean[:5])
    d = c.device()
    c.max_nodes = 4
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_OVERFLOW
    assert torch.equal(d["out"][:4], clean[:4]) and (d["out"][4] == 7.0).all()
    assert torch.equal(d["out"][5:9], clean[5:9])
    c.max_nodes = 5
    # offsets outside the arrays reach nothing
    d = c.device()
    d["cu"].copy_(torch.tensor([0, 5, 10 ** 6], dtype=torch.int32))
    c.run(d)
    assert int(d["st"].item()) & v4kv.V4KV_DEV_OVERFLOW
    assert torch.equal(d["out"], clean)
    # offsets that decrease: nothing is attended
    for cu in ([0, 9, 4], [3, 5, 2], [0, -1, 9]):
        d = c.device()
        d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        c.run(d)
        assert int(d["st"].item()) & v4kv.V4KV_DEV_OVERFLOW
        assert (d["out"] == 7.0).all()
    # a top-k entry the sequence does not hold
    c = TreeCase(871, [900], [3], 64, topk=50)
    d = c.device()
    c.run(d)
    clean = d["out"].clone()
    c.topk[1, 7] = -1
    d["topk"] = torch.from_numpy(c.topk).cuda()
    d["topk"][1, 7] = 225
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_BAD_INDEX
    c.check(d["out"])


def without(c, b, i, missing):
    """The oracle for a node whose entries on a page are left out."""
    lo = c.cu[b]
    depth = len(tree.family(c.parents[lo:c.cu[b + 1]], i)) - 1
    spb = 256 // c.ratio
    seen = np.arange(max(0, c.lens[b] + depth + 1 - c.W) // c.ratio)
    row = seen[seen // spb != missing].astype(np.int32)
    return tree.attend_node(c.q[lo + i], i, c.parents[lo:c.cu[b + 1]], c.k_tree[lo:c.cu[b + 1]], c.main.seq(b),
                            c.win.seq(b), c.lens[b], c.ratio, c.W, 1 / math.sqrt(512), topk_row=row)


@pytest.mark.parametrize("lens,counts,ratio,missing", [
    ([70000, 33000, 16600], [8, 3, 1], 128, 100),  # in a tile that every node sees
    ([70000, 33000, 16600], [8, 3, 1], 128, 272),  # in the last one
    ([70000, 33000, 16600], [2, 3, 1], 128, 100),
    ([3000, 700, 140], [8, 3, 1], 4, 3),
    ([3000, 700, 140], [8, 3, 1], 4, 11),
])
def test_missing_pages_and_scales_of_any_value(lens, counts, ratio, missing):
    from paged_compressed_kv_b200 import v4kv
    c = TreeCase(874 + missing, lens, counts, 64, ratio=ratio)
    r = synth.rng(10)
    c.main.scales[:] *= np.exp2(r.integers(-12, 4, c.main.scales.shape)).astype(np.float32)
    c.main.scales[r.random(c.main.scales.shape) < 0.1] = 0.0
    c.main.scales[r.random(c.main.scales.shape) < 0.2] *= -1.0
    d = c.device()
    c.run(d)
    assert int(d["st"].item()) == 0
    c.check(d["out"])
    clean = d["out"].clone()
    d["main"].block_table[0, missing] = 10 ** 6
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_BAD_PAGE
    n = counts[0]
    assert torch.equal(d["out"][n:], clean[n:])
    out = d["out"].float().cpu().numpy().astype(np.float64)
    for i in range(n):
        ref, mass = without(c, 0, i, missing)
        tol = (2.0 ** -9 + 2.0 ** -11) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mass.max()
        assert (np.abs(out[i] - ref) <= tol).all()


@pytest.mark.parametrize("lens,counts,ratio,missing", [
    ([3000, 700, 140], [8, 3, 1], 4, 3), ([3000, 700, 140], [8, 3, 1], 4, 11),
    ([3000, 700, 140], [2, 2, 1], 4, 3), ([70000, 33000, 16600], [8, 3, 1], 128, 100)])
def test_missing_pages_and_infinities_of_bf16_entries(lens, counts, ratio, missing):
    from paged_compressed_kv_b200 import v4kv
    c = TreeCase(879 + missing, lens, counts, 64, ratio=ratio, main_dtype="bf16")
    d = c.device()
    d["main"].block_table[0, missing] = -1
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_BAD_PAGE
    out = d["out"].float().cpu().numpy().astype(np.float64)
    n = counts[0]
    for i in range(n):
        ref, mass = without(c, 0, i, missing)
        tol = (2.0 ** -9 + 2.0 ** -11) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mass.max()
        assert (np.abs(out[i] - ref) <= tol).all()
    # an infinity, and a NaN, in an entry that every node sees
    clean = d["out"].clone()
    spb = 256 // ratio
    d["main"].data[int(c.main.bt[0, 1]), spb - 1, 9] = float("inf")
    d["main"].data[int(c.main.bt[1, 0]), spb - 1, 77] = float("nan")
    c.run(d)
    assert torch.isnan(d["out"][:n, :, 9]).all() and torch.isnan(d["out"][n:n + counts[1], :, 77]).all()
    assert torch.equal(d["out"][n + counts[1]:], clean[n + counts[1]:])


@pytest.mark.parametrize("heads,win_dtype,missing", [(64, "bf16", 0), (64, "fp8", 1), (10, "bf16", 1), (10, "fp8", 0)])
def test_missing_pages_of_the_window(heads, win_dtype, missing):
    """The tokens of a window page that is not there are left out, whatever the
    workspace held before; the other sequence is as it was."""
    from paged_compressed_kv_b200 import v4kv
    c = TreeCase(887 + heads, [300, 290], [4, 3], heads, win_dtype=win_dtype)
    d = c.device()
    c.run(d)
    clean = d["out"].clone()
    d["win"].block_table[0, missing] = -1
    d["ws"] = c.workspace(d)
    c.run(d)
    assert int(d["st"].item()) == v4kv.V4KV_DEV_BAD_PAGE
    assert torch.equal(d["out"][4:], clean[4:])
    out = d["out"].float().cpu().numpy().astype(np.float64)
    main, win = c.main.seq(0), c.win.seq(0)
    for i in range(4):
        fam = tree.family(c.parents[:4], i)
        pos = 300 + len(fam) - 1
        ents = list(range((pos + 1 - W) // 4))
        toks = [t for t in range(pos + 1 - W, 300) if t // 256 != missing]
        v = np.concatenate([c.k_tree[fam].astype(np.float64)] + [
            attention.gather(p["data"], p["scales"], p["dtype"], p["block_table_row"], at)
            for p, at in ((main, ents), (win, toks))])
        s = c.q[i].astype(np.float64) @ v.T / math.sqrt(512)
        w = np.exp(s - s.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        ref = rope_rotate(w @ v, pos, 1e6, 64, 448, inverse=True)
        mass = w @ np.abs(v)
        mass[:, 448:] = np.repeat(mass[:, 448:].reshape(heads, -1, 2).sum(axis=2), 2, axis=1)
        tol = (2.0 ** -9 + 2.0 ** -11) * mass + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mass.max()
        assert (np.abs(out[i] - ref) <= tol).all()


def test_scales_at_any_address():
    """Entry scales that begin 4, 8 and 12 bytes behind a 16-byte boundary."""
    c = TreeCase(876, [3000, 517], [5, 3], 64)
    d = c.device()
    c.run(d)
    c.check(d["out"])
    flat = d["main"].scales.reshape(-1)
    for off in (1, 2, 3):
        room = torch.full((flat.numel() + 4,), float("nan"), device="cuda")
        room[off:off + flat.numel()] = flat
        d["main"].scales = room[off:off + flat.numel()].view_as(d["main"].scales)
        d["out"].fill_(7.0)
        c.run(d)
        c.check(d["out"])
    assert int(d["st"].item()) == 0


@pytest.mark.parametrize("extra", [{}, dict(topk=200), dict(main_dtype="bf16"), dict(main_dtype="bf16", topk=200),
                                   dict(ratio=128)])
def test_pools_beyond_four_gigabytes(extra):
    """The same rows at the end of pools whose byte offsets do not fit 32 bits."""
    c = TreeCase(891, [2600, 700] if "ratio" not in extra else [30000, 17000], [7, 3], 64, **extra)
    d = c.device()
    c.run(d)
    clean = d["out"].clone()
    for name in ("main", "win"):
        pool = d[name]
        pages, page = pool.data.shape[0], pool.data[0].numel() * pool.data.element_size()
        more = (1 << 32) // page + 100
        data = torch.empty((more + pages,) + tuple(pool.data.shape[1:]), dtype=pool.data.dtype, device="cuda")
        data[more:] = pool.data
        pool.data = data
        if pool.scales is not None:
            scales = torch.empty(more + pages, pool.scales.shape[1], device="cuda")
            scales[more:] = pool.scales
            pool.scales = scales
        pool.block_table = torch.where(pool.block_table >= 0, pool.block_table + more, pool.block_table)
    d["out"].fill_(7.0)
    c.run(d)
    torch.cuda.synchronize()
    assert int(d["st"].item()) == 0
    assert torch.equal(d["out"], clean)


def test_graphs_that_share_a_workspace():
    """Two captured calls of different sequences with one workspace, replayed in turn."""
    c, e = TreeCase(877, [2000, 300], [6, 2], 64), TreeCase(878, [17000], [8], 64, ratio=128)
    d, f = c.device(), e.device()
    f["ws"] = d["ws"] = d["ws"] if d["ws"].numel() > f["ws"].numel() else f["ws"]
    c.run(d)
    ref = d["out"].clone()
    e.run(f)
    ref2 = f["out"].clone()
    graphs = []
    for case, dev in ((c, d), (e, f)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            case.run(dev)
    for _ in range(3):
        d["out"].fill_(0)
        f["out"].fill_(0)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d["out"], ref) and torch.equal(f["out"], ref2)


def test_host_refusals_that_need_a_device():
    from paged_compressed_kv_b200 import v4kv
    c = TreeCase(872, [300], [2], 64)
    d = c.device()
    small = dict(d, ws=d["ws"][:128])
    with pytest.raises(v4kv.V4KVError) as e:
        c.run(small)
    assert e.value.status == v4kv.V4KV_ERR_INVALID_ARG
    off = torch.empty(d["ws"].numel() + 16, dtype=torch.uint8, device="cuda")[16:]
    with pytest.raises(v4kv.V4KVError):
        c.run(dict(d, ws=off))
    assert (d["out"] == 7.0).all()


def test_no_nodes_at_all():
    c = TreeCase(873, [300, 20], [0, 0], 64)
    d = c.device()
    c.run(d)
    assert int(d["st"].item()) == 0


def test_streams_graphs_and_repeats_give_the_same_bits():
    c = TreeCase(880, [9000, 700, 33], [6, 1, 11], 64)
    e = TreeCase(881, [20000, 4000], [3, 8], 16, ratio=128)
    d, f = c.device(), e.device()
    c.run(d)
    e.run(f)
    ref, ref2 = d["out"].clone(), f["out"].clone()
    # two calls at once, each with its own workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        d["out"].fill_(0)
        f["out"].fill_(0)
        torch.cuda.synchronize()
        c.run(d, stream=s1)
        e.run(f, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(d["out"], ref) and torch.equal(f["out"], ref2)
    # captured, then replayed with other lengths, nodes and values in the same buffers
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(d)
        e.run(f)
    other = TreeCase(882, [8500, 200, 40], [4, 7, 7], 64)
    o = other.device()
    other.max_len, other.max_nodes = c.max_len, c.max_nodes
    o["ws"] = other.workspace(o)
    other.run(o)
    for name in ("q", "k_tree", "cu", "parents", "lens"):
        d[name].copy_(o[name])
    for p in ("main", "win"):
        n = min(d[p].data.shape[0], o[p].data.shape[0])
        d[p].data[:n].copy_(o[p].data[:n])
        if d[p].scales is not None:
            d[p].scales[:n].copy_(o[p].scales[:n])
        table = torch.full_like(d[p].block_table, -1)
        m = min(table.shape[1], o[p].block_table.shape[1])
        table[:, :m] = o[p].block_table[:, :m]
        assert int(table.max()) < n
        d[p].block_table.copy_(table)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["out"], o["out"]) and torch.equal(f["out"], ref2)
    assert int(d["st"].item()) == 0


# ------------------------------------------------------------------ verification

class VerifyCase:
    def __init__(self, seed, counts, vocab, shape="tree", draft=True, dtype=torch.float32, spread=2.0, pad=0):
        r = synth.rng(seed)
        self.counts, self.vocab, self.shape = list(counts), vocab, shape
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        n = self.N = int(self.cu[-1])
        self.parents = np.concatenate([make_parents(r, k, shape) for k in counts] + [[]]).astype(np.int32)
        x = synth.normal(r, (n, vocab), spread)
        y = x + synth.normal(r, (n, vocab), 0.7)

        def soft(v):
            e = np.exp(v - v.max(axis=1, keepdims=True))
            return torch.from_numpy((e / e.sum(axis=1, keepdims=True)).astype(np.float32)).to(dtype)

        self.target, self.draft = soft(x), soft(y) if draft else None
        q = soft(y).double().numpy()
        self.tokens = np.zeros(n, dtype=np.int32)
        for b, k in enumerate(counts):
            for i in range(1, k):
                row = q[self.cu[b] + self.parents[self.cu[b] + i]]
                self.tokens[self.cu[b] + i] = min(vocab - 1, int(np.searchsorted(np.cumsum(row), r.random() * row.sum())))
        self.u = r.random(n).astype(np.float32)
        self.s = r.random(len(counts)).astype(np.float32)
        self.pad, self.max_nodes = pad, max(max(counts), 1)

    def run(self):
        from paged_compressed_kv_b200 import v4kv

        def rows(t):
            wide = torch.full((self.N, self.vocab + self.pad), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, :self.vocab] = t.cuda()
            return wide[:, :self.vocab]

        i32 = dict(dtype=torch.int32, device="cuda")
        B = len(self.counts)
        path, n, nxt = torch.full((B, self.max_nodes), 99, **i32), torch.full((B,), 99, **i32), torch.full((B,), 99, **i32)
        st = torch.zeros(1, **i32)
        v4kv.v4kv_tree_verify(rows(self.target), torch.from_numpy(self.cu).cuda(), torch.from_numpy(self.parents).cuda(),
                              torch.from_numpy(self.tokens).cuda(), torch.from_numpy(self.u).cuda(),
                              torch.from_numpy(self.s).cuda(), self.max_nodes, path, n, nxt,
                              draft=rows(self.draft) if self.draft is not None else None, dev_status=st)
        return path.cpu().numpy(), n.cpu().numpy(), nxt.cpu().numpy(), int(st.item())

    def check(self):
        path, n, nxt, st = self.run()
        assert st == 0
        t = self.target.double().numpy()
        q = self.draft.double().numpy() if self.draft is not None else None
        for b, k in enumerate(self.counts):
            lo, hi = self.cu[b], self.cu[b + 1]
            if k == 0:
                assert n[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
                continue
            want, token = tree.verify(t[lo:hi], None if q is None else q[lo:hi], self.parents[lo:hi],
                                      self.tokens[lo:hi], self.u[lo:hi], self.s[b])
            assert list(path[b]) == want + [-1] * (self.max_nodes - len(want)), b
            assert n[b] == len(want) and nxt[b] == token, (b, nxt[b], token)
        return n


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 1000, 4099, 50257])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_matches_the_oracle(vocab, draft):
    n = VerifyCase(900 + vocab, [4, 1, 0, 9, 6, 6, 13, 6], vocab, draft=draft).check()
    if vocab == 1000 and draft:
        assert n.max() > 1  # paths of more than the root are among them


@pytest.mark.parametrize("shape,pad,dtype", [("chain", 0, torch.float32), ("star", 3, torch.float32),
                                             ("tree", 1, torch.bfloat16), ("star", 0, torch.bfloat16)])
def test_verify_shapes_strides_and_types(shape, pad, dtype):
    VerifyCase(930 + pad, [7, 30, 128, 3, 5], 517, shape=shape, pad=pad, dtype=dtype).check()
    VerifyCase(931 + pad, [7, 30, 128, 3, 5], 518, shape=shape, pad=pad, dtype=dtype, draft=False).check()


def test_verify_edges():
    from paged_compressed_kv_b200 import v4kv
    # equal draft and target: every child that is first asked is accepted
    c = VerifyCase(940, [6, 6, 6], 300, shape="chain")
    c.draft = c.target.clone()
    assert (c.check() == 6).all()
    # one-hot targets: the guess is taken exactly when it is the token
    c = VerifyCase(941, [4, 4], 64, shape="chain", draft=False)
    c.target = torch.zeros_like(c.target)
    c.target[torch.arange(8), torch.arange(8) + 3] = 1.0
    c.tokens = np.array([0, 3, 4, 60, 0, 7, 60, 9], dtype=np.int32)
    assert list(c.check()) == [3, 2]
    # numbers at the ends of the unit interval; duplicate children
    c = VerifyCase(942, [5, 5, 5], 40, shape="star", draft=False)
    c.tokens[:] = 11
    c.u[:], c.s[:] = 1.0 - 2.0 ** -24, [0.0, 1.0 - 2.0 ** -24, 1.0]
    c.check()
    c = VerifyCase(943, [5, 5, 5], 40, shape="star")
    c.u[:], c.s[:] = 1.0 - 2.0 ** -24, [0.0, 1.0 - 2.0 ** -24, 1.0]
    c.check()
    # a token outside the vocabulary, a row without mass, a second root
    c = VerifyCase(944, [3, 3], 40, shape="chain")
    c.tokens[1], c.tokens[5] = 40, -1
    path, n, nxt, st = c.run()
    assert st == v4kv.V4KV_DEV_BAD_INDEX and n[0] == 1
    c = VerifyCase(945, [2, 2], 40, shape="chain", draft=False)
    c.target[0] = 0.0
    path, n, nxt, st = c.run()
    assert st == v4kv.V4KV_DEV_BAD_PROB and nxt[0] == -1 and n[0] == 1 and nxt[1] >= 0
    c = VerifyCase(946, [3], 40, shape="forest")
    assert list(c.check()) == [1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch", [3, 90])
def test_verify_draws_at_the_ends_of_long_rows(batch, dtype):
    """Numbers at the ends of the unit interval, and rows whose mass is in a few
    values at the ends, the middle and behind a refused guess."""
    V = 65539
    c = VerifyCase(949, [2] * batch, V, dtype=dtype, draft=False, shape="chain")
    c.u[:], c.s[:] = 1.0 - 2.0 ** -24, np.tile([0.0, 0.5, 1.0 - 2.0 ** -24], batch // 3)
    c.check()
    c.target[:] = 0.0
    for i, at in enumerate([[0], [V - 1], [0, V - 1], [1, 2, V - 3], [V // 2], [0, V // 3, V - 2]]):
        c.target[i, at] = torch.tensor([0.5, 0.25, 0.25][:len(at)], dtype=dtype)
    c.target[6:] = c.target[:6].repeat(batch // 3, 1)[:2 * batch - 6]
    c.tokens[:] = V - 1
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_takes_values_that_are_not_positive_as_zero(dtype):
    for draft in (True, False):
        c = VerifyCase(947, [9, 6, 30, 4], 211, dtype=dtype, draft=draft)
        r = synth.rng(948)
        for t in (c.target, c.draft)[:1 + draft]:
            at = torch.from_numpy(r.random(tuple(t.shape)))
            t[at < 0.3] *= -1.0
            t[at > 0.9] = float("nan")
        c.check()


def test_verify_and_gather_captured_and_at_once():
    """Replays with other values in the same buffers, and calls on two streams."""
    from paged_compressed_kv_b200 import v4kv
    i32 = dict(dtype=torch.int32, device="cuda")

    def prepare(c):
        B, n = len(c.counts), c.N
        t = dict(target=c.target.cuda(), draft=c.draft.cuda(), cu=torch.from_numpy(c.cu).cuda(),
                 parents=torch.from_numpy(c.parents).cuda(), tokens=torch.from_numpy(c.tokens).cuda(),
                 u=torch.from_numpy(c.u).cuda(), s=torch.from_numpy(c.s).cuda(), path=torch.zeros(B, c.max_nodes, **i32),
                 n=torch.zeros(B, **i32), nxt=torch.zeros(B, **i32), x=torch.arange(n * 8.0, device="cuda").view(n, 8),
                 gate=torch.arange(float(n), device="cuda"), cuo=torch.zeros(B + 1, **i32))
        t["x"] = t["x"].to(torch.bfloat16)
        t["xo"], t["go"] = torch.zeros_like(t["x"]), torch.zeros_like(t["gate"])
        return t

    def run(c, t, stream=None):
        v4kv.v4kv_tree_verify(t["target"], t["cu"], t["parents"], t["tokens"], t["u"], t["s"], c.max_nodes, t["path"],
                              t["n"], t["nxt"], draft=t["draft"], stream=stream)
        v4kv.v4kv_tree_gather(t["x"], t["gate"], t["cu"], t["path"], t["n"], t["xo"], t["go"], t["cuo"], stream=stream)

    outs = ("path", "n", "nxt", "xo", "go", "cuo")
    cases = [VerifyCase(seed, [6] * 40, 5003) for seed in (970, 971)]
    first, second = (prepare(c) for c in cases)
    for c, t in zip(cases, (first, second)):
        run(c, t)
    want = [{k: t[k].clone() for k in outs} for t in (first, second)]
    assert not torch.equal(want[0]["nxt"], want[1]["nxt"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for t in (first, second):
            for k in outs:
                t[k].zero_()
        torch.cuda.synchronize()
        for c, t, s in zip(cases, (first, second), streams):
            run(c, t, stream=s)
        torch.cuda.synchronize()
        for t, w in zip((first, second), want):
            assert all(torch.equal(t[k], w[k]) for k in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(cases[0], first)
    for k in set(first) - set(outs):
        first[k].copy_(second[k])
    for k in outs:
        first[k].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], want[1][k]) for k in outs)


@pytest.mark.parametrize("batch", [5, 40, 90])  # clusters of 8, 4 and 2 blocks
def test_verify_while_its_blocks_start_apart(batch):
    """Blocks of a cluster start as a busy GPU frees their places, and some
    clusters leave at once: every repeat gives the oracle's tokens."""
    c = VerifyCase(960 + batch, [7, 0, 5, 1, 0][:5] * (batch // 5), 4099)
    busy, side = torch.randn(4096, 4096, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(side):
            for _ in range(3):
                busy.sum(dim=1)
                busy.square()
        c.check()
    torch.cuda.synchronize()


# ------------------------------------------------------------------ packing and a whole step

@pytest.mark.parametrize("dim,per_channel", [(8, False), (512, False), (512, True), (1024, True), (200, True)])
def test_gather_packs_the_accepted_rows(dim, per_channel):
    from paged_compressed_kv_b200 import v4kv
    r = synth.rng(950 + dim)
    counts = [5, 0, 1, 30, 2, 128] + [3] * 300
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    N, B, most = int(cu[-1]), len(counts), max(counts)
    path, n = np.full((B, most), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b, k in enumerate(counts):
        n[b] = r.integers(1, k + 1) if k else 0
        path[b, :n[b]] = np.sort(r.permutation(k)[:n[b]])
    x = synth.bf16_tensor(synth.normal(r, (N, dim))).cuda()
    gate = torch.from_numpy(synth.normal(r, (N, dim) if per_channel else N)).cuda()
    total = int(n.sum())
    rows = torch.from_numpy(np.concatenate([cu[b] + path[b, :n[b]] for b in range(B)])).long().cuda()
    for cap in (N, total, total - 7):
        xo = torch.full((cap, dim), 3.0, dtype=torch.bfloat16, device="cuda")
        go = torch.full((cap, dim) if per_channel else (cap,), 3.0, device="cuda")
        cuo = torch.full((B + 1,), -5, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        v4kv.v4kv_tree_gather(x, gate, torch.from_numpy(cu).cuda(), torch.from_numpy(path).cuda(),
                              torch.from_numpy(n).cuda(), xo, go, cuo, dev_status=st)
        m = min(cap, total)
        assert torch.equal(xo[:m], x[rows[:m]]) and torch.equal(go[:m], gate[rows[:m]])
        assert (xo[m:] == 3.0).all() and (go[m:] == 3.0).all()
        want = np.minimum(np.concatenate([[0], np.cumsum(n)]), cap)
        assert (cuo.cpu().numpy() == want).all()
        assert int(st.item()) == (v4kv.V4KV_DEV_OVERFLOW if cap < total else 0)
    path[3, 0] = 30
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    xo = torch.full((N, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    go = torch.full((N, dim) if per_channel else (N,), 3.0, device="cuda")
    v4kv.v4kv_tree_gather(x, gate, torch.from_numpy(cu).cuda(), torch.from_numpy(path).cuda(),
                          torch.from_numpy(n).cuda(), xo, go, cuo, dev_status=st)
    assert int(st.item()) == v4kv.V4KV_DEV_BAD_INDEX
    at = int(n[:3].sum())
    assert not xo[at].any() and not go[at].any() and torch.equal(xo[at + 1:total], x[rows[at + 1:]])


def test_a_speculative_step_equals_appending_the_accepted_tokens():
    """The operators together, as a serving loop runs them and without reading
    anything back: rotate q and K of the drafted nodes, attend, verify, pack,
    append. The cache afterwards is bit for bit the one that appending the
    accepted tokens gives, and the next step's attention agrees with it."""
    from paged_compressed_kv_b200 import PagedPool, Rope, v4kv
    r = synth.rng(960)
    B, H, ratio, T, vocab = 3, 8, 4, 6, 97
    lens = [517, 130, 255]
    dev = dict(device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def pools():
        main = PagedPool(data=torch.zeros(3 * B, 64, 512, dtype=torch.uint8, **dev),
                         scales=torch.zeros(3 * B, 64, **dev),
                         block_table=torch.arange(3 * B, **i32).view(B, 3).flip(1).contiguous())
        win = PagedPool(data=torch.zeros(3 * B, 256, 512, dtype=torch.bfloat16, **dev),
                        block_table=torch.arange(3 * B, **i32).view(3, B).t().contiguous())
        state = (torch.zeros(B, ratio, 512, dtype=torch.bfloat16, **dev), torch.zeros(B, ratio, **dev))
        return main, win, state

    bias = torch.from_numpy(synth.normal(r, ratio, 0.5)).cuda()
    prompt = synth.bf16_tensor(synth.normal(r, (sum(lens), 512))).cuda()
    pgate = torch.from_numpy(synth.normal(r, sum(lens))).cuda()
    parents = torch.tensor(make_parents(r, T, "tree") * B, **i32)
    cu = torch.arange(B + 1, **i32) * T
    x = synth.bf16_tensor(synth.normal(r, (B * T, 512))).cuda()
    gate = torch.from_numpy(synth.normal(r, B * T)).cuda()
    q = torch.from_numpy(synth.normal(r, (B * T, H, 512))).cuda()
    depth = torch.tensor([len(tree.family(parents[:T].tolist(), i)) - 1 for i in range(T)] * B, **i32)
    target = torch.softmax(torch.from_numpy(synth.normal(r, (B * T, vocab), 3.0)).cuda(), -1)
    tokens = target.argmax(-1).to(torch.int32).view(B, T).gather(1, parents.view(B, T).clamp(min=0).long()).view(-1).contiguous()
    u, s = torch.from_numpy(r.random(B * T).astype(np.float32)).cuda() * 0.5, torch.from_numpy(r.random(B).astype(np.float32)).cuda()
    st = torch.zeros(1, **i32)

    def append(main, win, state, x, gate, cu_seq, start):
        v4kv.v4kv_compress_append(x, gate, cu_seq, start, bias, ratio, state[0], state[1], main, None, None, window=win,
                                  window_len=W, rope=Rope(), dev_status=st)

    def attend(main, win, L, nodes_q, cu_n, par, k_rows, n):
        out = torch.empty(nodes_q.shape, dtype=torch.bfloat16, **dev)
        size = v4kv.v4kv_tree_workspace_size(B, H, nodes_q.shape[0], n, 700, ratio, W, 0, main.dtype_code)
        v4kv.v4kv_tree_attention(nodes_q, cu_n, par, k_rows, main, win, L, n, 700, ratio, W, out,
                                 torch.empty(max(size, 256), dtype=torch.uint8, **dev), dev_status=st)
        return out

    def rotate(v, pos):
        out = torch.empty(v.shape, dtype=torch.bfloat16, **dev)
        v4kv.v4kv_qk_prepare(v.contiguous(), pos, out, rope=Rope())
        return out

    start = torch.tensor(lens, **i32)
    zero = torch.zeros(B, **i32)
    cu_p = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), **i32)
    main, win, state = pools()
    append(main, win, state, prompt, pgate, cu_p, zero)
    pos = start.repeat_interleave(T) + depth
    out = attend(main, win, start, rotate(q, pos), cu, parents, rotate(x.float().view(-1, 1, 512), pos).view(-1, 512), T)
    path, n_path, nxt = torch.empty(B, T, **i32), torch.empty(B, **i32), torch.empty(B, **i32)
    v4kv.v4kv_tree_verify(target, cu, parents, tokens, u, s, T, path, n_path, nxt, dev_status=st)
    xo, go, cuo = torch.zeros_like(x), torch.zeros_like(gate), torch.empty(B + 1, **i32)
    v4kv.v4kv_tree_gather(x, gate, cu, path, n_path, xo, go, cuo, dev_status=st)
    append(main, win, state, xo, go, cuo, start)   # all of xo's rows, as the host does not know the count
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.isfinite(out.float()).all()
    n = n_path.tolist()
    assert max(n) > 1, n  # something was accepted
    # the same tokens appended directly
    main2, win2, state2 = pools()
    append(main2, win2, state2, prompt, pgate, cu_p, zero)
    rows = torch.cat([cu[b] + path[b, :n[b]] for b in range(B)]).long()
    append(main2, win2, state2, x[rows].contiguous(), gate[rows].contiguous(),
           torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32), start)
    assert torch.equal(main.data, main2.data) and torch.equal(main.scales, main2.scales)
    assert torch.equal(win.data, win2.data)
    # an accepted path's last node equals a root attending the appended cache one token earlier:
    # the same items, in the window instead of the tree
    last = torch.stack([cu[b] + path[b, n[b] - 1] for b in range(B)]).long()
    one = attend(main, win, start + n_path - 1, rotate(q, pos)[last].contiguous(), torch.arange(B + 1, **i32),
                 torch.full((B,), -1, **i32), rotate(x.float().view(-1, 1, 512), pos).view(-1, 512)[last].contiguous(), 1)
    a, b = out[last].float(), one.float()
    assert float((a - b).abs().max()) <= 2e-2 * float(b.abs().max())
    assert int(st.item()) == 0
