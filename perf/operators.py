"""The speculative-decoding operators: their cases, plain forms and exact values.

Three operators over the paged, compressed cache take a batch of drafted token
trees through one step:

  tree_attention  every drafted node attends to the committed cache (compressed
                  entries or its own top-k of them, and the raw-token window)
                  and to its ancestors in the tree;
  tree_verify     the drafted tokens are checked against the target's
                  probabilities with given random numbers, giving the accepted
                  path and the next token;
  tree_gather     the accepted nodes' raw rows and gates are packed in the form
                  that the cache's append takes.

A tree is a list of nodes in which every parent comes before its children;
``parents`` holds the parent's index within the sequence, -1 for a root. Node i
of a sequence with L committed tokens sits at position L + depth(i).

With ``own`` false, ``run`` computes the operators from elementary torch
operations; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DIM = 512          # shared K = V dims
WINDOW = 128       # raw-token window
BLOCK = 256        # raw tokens per page
THETA, ROPE_DIM, ROPE_OFFSET = 1e6, 64, 448
SCALE = 1.0 / math.sqrt(DIM)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short conversation, a handful of drafted tokens, eight heads and
        # bf16 entries: launch latency
        dict(name="attend-tiny", op="attend", batch=1, nodes=5, ragged=False, chain=False, heads=8, ratio=4,
             entries_bf16=True, dist="uniform", lo=1024, hi=1024, topk=0, q_fp32=False),
        # a full serving batch, 4K to 64K tokens of context, all c4a entries
        dict(name="attend-c4a-b64", op="attend", batch=64, nodes=8, ragged=False, chain=False, heads=64, ratio=4,
             entries_bf16=False, dist="uniform", lo=4096, hi=65536, topk=0, q_fp32=False),
        # long contexts in a c128a layer, 128K to 1M tokens
        dict(name="attend-c128a-b32", op="attend", batch=32, nodes=16, ragged=False, chain=False, heads=64, ratio=128,
             entries_bf16=False, dist="log", lo=131072, hi=1000000, topk=0, q_fp32=False),
        # c4a layers with an indexer: each node reads its own 512 entries
        dict(name="attend-top512-b32", op="attend", batch=32, nodes=6, ragged=False, chain=True, heads=64, ratio=4,
             entries_bf16=False, dist="uniform", lo=1024, hi=262144, topk=512, q_fp32=False),
        # one long conversation and a wide tree: the entries are split over the GPU
        dict(name="attend-long-b1", op="attend", batch=1, nodes=31, ragged=False, chain=False, heads=64, ratio=4,
             entries_bf16=False, dist="uniform", lo=131001, hi=131001, topk=0, q_fp32=False),
        # short, odd lengths, trees of different sizes (some of one node), fp32 queries
        dict(name="attend-ragged-h16", op="attend", batch=13, nodes=11, ragged=True, chain=False, heads=16, ratio=4,
             entries_bf16=False, dist="log", lo=1, hi=6001, topk=0, q_fp32=True),
        # one sequence, a short chain of drafts sampled from the draft's distribution
        dict(name="verify-chain-b1", op="verify", batch=1, nodes=5, chain=True, vocab=32001, draft=True),
        # a batch of trees whose children were sampled from the draft's distribution
        dict(name="verify-tree-b32", op="verify", batch=32, nodes=12, chain=False, vocab=131072, draft=True),
        # a serving batch of chains whose drafts are fixed guesses (no draft distribution)
        dict(name="verify-guess-b64", op="verify", batch=64, nodes=6, chain=True, vocab=131072, draft=False),
        # one sequence's accepted rows, a gate per token
        dict(name="gather-b1", op="gather", batch=1, nodes=5, dim=512, gate_dim=1),
        # a large batch with a gate per channel
        dict(name="gather-b128", op="gather", batch=128, nodes=64, dim=512, gate_dim=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "gather"])
    if op == "attend":
        topk = rng.choice([0, 0, rng.randint(1, 700)])
        heads = rng.choice([8, 16, 24, 64, 64, 128])
        ratio = 4 if topk else rng.choice([4, 128])
        batch = _log(rng, 1, 48)
        nodes = max(1, min(_log(rng, 1, 40), 18000 // (heads * batch)))
        hi = _log(rng, 2, 60000 if ratio == 4 else 900000)
        return dict(op=op, batch=batch, nodes=nodes, ragged=rng.random() < 0.5, chain=rng.random() < 0.4, heads=heads,
                    ratio=ratio, entries_bf16=rng.random() < 0.25, dist=rng.choice(["uniform", "log"]),
                    lo=max(1, hi // rng.randint(1, 16)), hi=hi, topk=topk, q_fp32=rng.random() < 0.3)
    if op == "verify":
        return dict(op=op, batch=_log(rng, 1, 40), nodes=_log(rng, 1, 12), chain=rng.random() < 0.5,
                    vocab=_log(rng, 50, 131072), draft=rng.random() < 0.6)
    return dict(op=op, batch=_log(rng, 1, 128), nodes=_log(rng, 1, 64), dim=8 * rng.randint(1, 128),
                gate_dim=rng.choice([1, 0]))


def _lengths(case):
    """The committed lengths: quantiles of the case's distribution, so that a
    case's work does not depend on the seed."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    at = [(i + 0.5) / n for i in range(n)]
    if case["dist"] == "log":
        return [int(round(lo * (hi / lo) ** u)) for u in at]
    return [int(round(lo + (hi - lo) * u)) for u in at]


def _counts(case):
    """Nodes of each sequence; a ragged batch runs from one node to the most."""
    n, most = case["batch"], case["nodes"]
    return [1 + (i * 7) % most for i in range(n)] if case.get("ragged") else [most] * n


# ------------------------------------------------------------------ inputs

def _generators(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    h = torch.Generator()
    h.manual_seed(1000003 * seed + 29)
    return g, h


def _trees(counts, chain, h):
    """Parents of every sequence's nodes: a chain, or a tree that widens with
    depth as a drafter's does."""
    parents = []
    for n in counts:
        u = torch.rand(max(n, 1), generator=h).tolist()
        for i in range(n):
            if i == 0:
                parents.append(-1)
            elif chain:
                parents.append(i - 1)
            else:
                lo, hi = (i - 1) // 4, (i - 1) // 2
                parents.append(lo + int(u[i] * (hi - lo + 1)))
    return parents


def _offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(first, blocks, h):
    """A shuffled block table [batch, most blocks]; blocks before ``first`` have no page."""
    total = sum(n - f for f, n in zip(first, blocks))
    perm = torch.randperm(total, generator=h)
    table = torch.full((len(blocks), max(blocks + [1])), -1, dtype=torch.int64)
    at = 0
    for b, (f, n) in enumerate(zip(first, blocks)):
        table[b, f:n] = perm[at:at + n - f]
        at += n - f
    return table.to(torch.int32).cuda(), max(total, 1)


def _prepare_attend(case, seed):
    g, h = _generators(seed)
    ratio, heads = case["ratio"], case["heads"]
    order = torch.randperm(case["batch"], generator=h).tolist()
    lens = [_lengths(case)[i] for i in order]
    counts = _counts(case)
    cu = _offsets(counts)
    slots = BLOCK // ratio
    entries = [-(-n // ratio) for n in lens]
    table, pages = _pages([0] * len(lens), [-(-e // slots) for e in entries], h)
    wtable, wpages = _pages([max(0, n - WINDOW) // BLOCK for n in lens], [-(-n // BLOCK) for n in lens], h)
    s = dict(case=case, ratio=ratio, slots=slots, max_nodes=max(counts), max_len=max(lens))
    s["table"], s["wtable"] = table, wtable
    shape = (pages, slots, DIM)
    if case["entries_bf16"]:
        s["data"] = torch.randn(shape, generator=g, device="cuda").mul_(0.5).to(torch.bfloat16)
        s["scales"] = None
    else:
        x = torch.randn(shape, generator=g, device="cuda").mul_(112.0).clamp_(-448.0, 448.0)
        s["data"] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        s["scales"] = (torch.rand(shape[:2], generator=g, device="cuda") + 0.5) * (0.5 / 112.0)
        del x
    s["window"] = torch.randn((wpages, BLOCK, DIM), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((cu[-1], heads, DIM), generator=g, device="cuda") * 1.5
    s["q"] = q if case["q_fp32"] else q.to(torch.bfloat16)
    s["k_tree"] = torch.randn((cu[-1], DIM), generator=g, device="cuda").to(torch.bfloat16)
    s["parents"] = _int(_trees(counts, case["chain"], h))
    s["cu"], s["lens"] = _int(cu), _int(lens)
    s["topk"] = None
    if case["topk"]:
        # an indexer's choice for each node: distinct visible entries, -1 behind them where there are fewer
        k = case["topk"]
        seq = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
        seen = (torch.tensor(lens) + 1 - WINDOW).clamp(min=0) // ratio
        step = torch.rand((cu[-1], k), generator=h) + 0.05
        at = step.cumsum(1)
        n = seen[seq].double()
        pick = (at.double() / (at[:, -1:] + 0.5) * n[:, None]).floor().to(torch.int64)
        new = torch.ones_like(pick, dtype=torch.bool)
        new[:, 1:] = pick[:, 1:] > pick[:, :-1]
        pick = torch.where(new & (n[:, None] > 0), pick, torch.full_like(pick, -1))
        s["topk"] = pick.to(torch.int32).cuda()
    s["out"] = torch.zeros((cu[-1], heads, DIM), dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_verify(case, seed):
    g, h = _generators(seed)
    batch, nodes, vocab = case["batch"], case["nodes"], case["vocab"]
    n = batch * nodes
    parents = _int(_trees([nodes] * batch, case["chain"], h))
    rows = torch.arange(n, device="cuda")
    up = (rows // nodes * nodes + parents).clamp(min=0)  # the parent's row (a root's own is not used)
    up = torch.where(parents < 0, rows, up)
    logits = torch.randn((n, vocab), generator=g, device="cuda") * 2.5
    s = dict(case=case, max_nodes=nodes, parents=parents, cu=_int([i * nodes for i in range(batch + 1)]))
    s["target"] = torch.softmax(logits, -1)
    logits += torch.randn((n, vocab), generator=g, device="cuda") * 0.7
    draft = torch.softmax(logits, -1)
    if case["draft"]:
        s["draft"] = draft
        at = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        sums = draft[up].double().cumsum(-1)
        s["tokens"] = torch.searchsorted(sums, at[:, None] * sums[:, -1:], right=True)[:, 0].clamp(max=vocab - 1).to(torch.int32)
    else:
        s["draft"] = None
        rank = (rows - up - 1).clamp(min=0) % 4  # siblings guess different tokens
        best = draft.topk(min(4, vocab), -1).indices[up]
        s["tokens"] = best.gather(1, rank[:, None] % best.shape[1])[:, 0].to(torch.int32)
    del logits, draft
    s["accept"] = torch.rand(n, generator=g, device="cuda")
    s["sample"] = torch.rand(batch, generator=g, device="cuda")
    s["path"] = torch.zeros((batch, nodes), dtype=torch.int32, device="cuda")
    s["n_path"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
    s["next"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
    return s


def _prepare_gather(case, seed):
    g, h = _generators(seed)
    batch, dim = case["batch"], case["dim"]
    width = case["gate_dim"] if case["gate_dim"] else dim
    counts = _counts(dict(case, ragged=batch > 1))
    cu = _offsets(counts)
    parents = _trees(counts, False, h)
    ends = torch.rand(batch, generator=h).tolist()
    path = torch.full((batch, max(counts)), -1, dtype=torch.int32)
    length = []
    for b, n in enumerate(counts):
        i, chain = int(ends[b] * n), []
        while i >= 0:
            chain.append(i)
            i = parents[cu[b] + i]
        path[b, :len(chain)] = torch.tensor(chain[::-1], dtype=torch.int32)
        length.append(len(chain))
    s = dict(case=case, max_nodes=max(counts), cu=_int(cu), path=path.cuda(), n_path=_int(length))
    s["x"] = torch.randn((cu[-1], dim), generator=g, device="cuda").to(torch.bfloat16)
    s["gate"] = torch.randn((cu[-1], width) if width > 1 else (cu[-1],), generator=g, device="cuda")
    s["x_out"], s["gate_out"] = torch.zeros_like(s["x"]), torch.zeros_like(s["gate"])
    s["cu_out"] = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    return {"attend": _prepare_attend, "verify": _prepare_verify, "gather": _prepare_gather}[case["op"]](case, seed)


# ------------------------------------------------------------------ plain forms

def _nodes(s, batch):
    """Per node: its sequence and index in it, its depth, and which nodes of the
    same sequence are its ancestors or itself [nodes, most nodes]."""
    cu, parents, most = s["cu"].long(), s["parents"].long(), s["max_nodes"]
    rows = torch.arange(parents.numel(), device="cuda")
    seq = torch.searchsorted(cu, rows, right=True) - 1
    at = rows - cu[seq]
    # with parents before children, I - (parent matrix) is unit lower triangular
    # and its inverse is the sum of the parent matrix's powers: one where a node
    # is an ancestor of the row's
    step = torch.eye(most, device="cuda").repeat(batch, 1, 1)
    child = parents >= 0
    step[seq[child], at[child], parents[child]] = -1.0
    eye = torch.eye(most, device="cuda").expand(batch, most, most)
    up = torch.linalg.solve_triangular(step, eye, upper=False, unitriangular=True)[seq, at] > 0.5
    return seq, at, up.sum(1) - 1, up


def _rows(data, scales, table, index, slots):
    """Values of logical indices [batch, n] through the block table, in 32 bits."""
    page = table.long().gather(1, (index // slots).clamp(min=0, max=table.shape[1] - 1)).clamp(min=0)
    slot = page * slots + index.clamp(min=0) % slots
    x = data.view(-1, data.shape[-1])[slot]
    if scales is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * scales.view(-1)[slot][..., None]


def _plain_attend(s):
    case, ratio, slots = s["case"], s["ratio"], s["slots"]
    lens, batch, heads, most = s["lens"].long(), s["lens"].numel(), s["case"]["heads"], s["max_nodes"]
    seq, at, depth, up = _nodes(s, batch)
    n = seq.numel()
    end = lens[seq] + depth + 1                     # the tokens up to and with the node
    # the batch padded to the longest: values of entries, window tokens and nodes
    q = torch.zeros((batch, most, heads, DIM), device="cuda")
    q[seq, at] = s["q"].float()
    k_tree = torch.zeros((batch, most, DIM), device="cuda")
    k_tree[seq, at] = s["k_tree"].float()
    w0 = (lens + 1 - WINDOW).clamp(min=0)
    wi = w0[:, None] + torch.arange(WINDOW, device="cuda")
    win = _rows(s["window"], None, s["wtable"], wi.clamp(max=max(0, s["wtable"].shape[1] * BLOCK - 1)), BLOCK)
    near = torch.cat([win, k_tree], 1)
    seen = torch.zeros((batch, most, WINDOW + most), dtype=torch.bool, device="cuda")
    tok = wi[seq]
    seen[seq, at, :WINDOW] = (tok >= end[:, None] - WINDOW) & (tok < lens[seq][:, None])
    seen[seq, at, WINDOW:] = up
    score = torch.matmul(q.view(batch, most * heads, DIM), near.transpose(1, 2)).view(batch, most, heads, -1) * SCALE
    score = score.masked_fill(~seen[:, :, None], -math.inf)
    if s["topk"] is not None:
        pick = s["topk"].long()
        far = _rows(s["data"], s["scales"], s["table"][seq], pick, slots)          # [nodes, k, DIM]
        fs = torch.matmul(q[seq, at], far.transpose(1, 2)) * SCALE                 # [nodes, heads, k]
        fs = fs.masked_fill((pick < 0)[:, None], -math.inf)
        both = torch.cat([score[seq, at], fs], -1)
        p = torch.exp(both - both.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = torch.matmul(p[..., -pick.shape[1]:], far)
        p_near = torch.zeros_like(score)
        p_near[seq, at] = p[..., :WINDOW + most]
        o = o + torch.matmul(p_near.view(batch, most * heads, -1), near).view(batch, most, heads, DIM)[seq, at]
    else:
        entries = max(1, (s["max_len"] + most - WINDOW) // ratio)
        j = torch.arange(entries, device="cuda").expand(batch, entries)
        far = _rows(s["data"], s["scales"], s["table"], j, slots)
        visible = torch.zeros((batch, most, entries), dtype=torch.bool, device="cuda")
        visible[seq, at] = j[seq] < ((end - WINDOW).clamp(min=0) // ratio)[:, None]
        fs = torch.matmul(q.view(batch, most * heads, DIM), far.transpose(1, 2)).view(batch, most, heads, -1) * SCALE
        fs = fs.masked_fill(~visible[:, :, None], -math.inf)
        top = torch.maximum(score.amax(-1), fs.amax(-1))[..., None]
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)            # a padded node sees nothing
        pn, pf = torch.exp(score - top), torch.exp(fs - top)
        total = (pn.sum(-1) + pf.sum(-1))[..., None]
        o = torch.matmul(pf.view(batch, most * heads, -1), far) + torch.matmul(pn.view(batch, most * heads, -1), near)
        o = (o.view(batch, most, heads, DIM) / total)[seq, at]
    # the inverse rotation at the node's position, its angles in 64 bits
    pair = torch.arange(ROPE_DIM // 2, device="cuda", dtype=torch.float64)
    angle = (lens[seq] + depth).double()[:, None] * THETA ** (-2.0 * pair / ROPE_DIM)
    c, t = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = o[..., ROPE_OFFSET::2], o[..., ROPE_OFFSET + 1::2]
    o = torch.cat([o[..., :ROPE_OFFSET], torch.stack([a * c + b * t, b * c - a * t], -1).view(n, heads, ROPE_DIM)], -1)
    return o.to(torch.bfloat16)


def _plain_verify(s):
    batch, nodes = s["case"]["batch"], s["max_nodes"]
    target, draft, vocab = s["target"], s["draft"], s["case"]["vocab"]
    first = s["cu"][:-1].long()
    parents, tokens = s["parents"].view(batch, nodes).long(), s["tokens"].view(batch, nodes).long()
    u = s["accept"].view(batch, nodes).double()
    every = torch.arange(batch, device="cuda")
    now = torch.zeros(batch, dtype=torch.long, device="cuda")       # the last accepted node
    path = torch.full((batch, nodes), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    n_path = torch.ones(batch, dtype=torch.long, device="cuda")
    left = target[first].double()                                    # what is left of the target's row there
    mass = torch.ones(batch, dtype=torch.float64, device="cuda")
    taken = torch.zeros(batch, dtype=torch.float64, device="cuda")  # how often the draft's row was taken from it
    for i in range(1, nodes):
        asked = parents[:, i] == now
        x = tokens[:, i]
        have = left[every, x]
        q = draft[first + now, x].double() if draft is not None else torch.ones_like(have)
        yes = asked & (u[:, i] * q * mass < have)
        no = asked & ~yes
        # refused: what is left is the target's row less the draft's, or without the token
        if draft is not None:
            taken = torch.where(no, taken + mass, taken)
            less = (target[first + now].double() - taken[:, None] * draft[first + now].double()).clamp(min=0)
            left = torch.where(no[:, None], less, left)
            mass = torch.where(no, less.sum(-1), mass)
        else:
            mass = torch.where(no, mass - have, mass)
            left[every[no], x[no]] = 0.0
        now = torch.where(yes, i, now)
        path[every[yes], n_path[yes]] = i
        n_path = n_path + yes
        left = torch.where(yes[:, None], target[first + i].double(), left)
        mass, taken = torch.where(yes, 1.0, mass), torch.where(yes, 0.0, taken)
    # the next token, from what is left of the last accepted node's row (all of it if nothing is)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, target[first + now].double())
    sums = left.cumsum(-1)
    token = (sums <= s["sample"].double()[:, None] * sums[:, -1:]).sum(-1)
    last = vocab - 1 - (left.flip(-1) > 0).to(torch.int32).argmax(-1)
    return {"path": path, "n_path": n_path.to(torch.int32), "next": torch.minimum(token, last).to(torch.int32)}


def _plain_gather(s):
    path, n = s["path"].long(), s["n_path"].long()
    cu = torch.zeros(n.numel() + 1, dtype=torch.long, device="cuda")
    cu[1:] = n.cumsum(0)
    used = torch.arange(path.shape[1], device="cuda") < n[:, None]
    rows = (s["cu"][:-1].long()[:, None] + path)[used]
    x, gate = torch.zeros_like(s["x"]), torch.zeros_like(s["gate"])
    x[:rows.numel()], gate[:rows.numel()] = s["x"][rows], s["gate"][rows]
    return {"x": x, "gate": gate, "cu": cu.to(torch.int32)}


# ------------------------------------------------------------------ the library's calls

def _own_attend(s):
    from paged_compressed_kv_b200 import PagedPool, v4kv
    case = s["case"]
    if "call" not in s:  # what a program sets up once: the pools' descriptions and the scratch
        main = PagedPool(data=s["data"], block_table=s["table"], scales=s["scales"])
        window = PagedPool(data=s["window"], block_table=s["wtable"])
        size = v4kv.v4kv_tree_workspace_size(case["batch"], case["heads"], s["q"].shape[0], s["max_nodes"], s["max_len"],
                                             s["ratio"], WINDOW, case["topk"], main.dtype_code)
        s["call"] = main, window, torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    main, window, scratch = s["call"]
    v4kv.v4kv_tree_attention(s["q"], s["cu"], s["parents"], s["k_tree"], main, window, s["lens"], s["max_nodes"],
                             s["max_len"], s["ratio"], WINDOW, s["out"], scratch, topk=s["topk"])
    return s["out"]


def _own_verify(s):
    from paged_compressed_kv_b200 import v4kv
    v4kv.v4kv_tree_verify(s["target"], s["cu"], s["parents"], s["tokens"], s["accept"], s["sample"], s["max_nodes"],
                          s["path"], s["n_path"], s["next"], draft=s["draft"])
    return {"path": s["path"], "n_path": s["n_path"], "next": s["next"]}


def _own_gather(s):
    from paged_compressed_kv_b200 import v4kv
    v4kv.v4kv_tree_gather(s["x"], s["gate"], s["cu"], s["path"], s["n_path"], s["x_out"], s["gate_out"], s["cu_out"])
    return {"x": s["x_out"], "gate": s["gate_out"], "cu": s["cu_out"]}


def run(state):
    plain = {"attend": _plain_attend, "verify": _plain_verify, "gather": _plain_gather}
    calls = {"attend": _own_attend, "verify": _own_verify, "gather": _own_gather}
    return (calls if own else plain)[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "attend":
        heads, width = case["heads"], 2 * DIM if case["entries_bf16"] else DIM + 4
        size = flops = 0
        for length, nodes in zip(_lengths(case), _counts(case)):
            seen = max(0, length + 1 - WINDOW) // case["ratio"]
            rows = nodes * heads
            per_node = min(case["topk"], seen) if case["topk"] else seen
            read = min(per_node * nodes, seen)
            tokens = min(length, WINDOW - 1)
            size += read * width + (tokens + nodes) * 2 * DIM + rows * DIM * ((4 if case["q_fp32"] else 2) + 2)
            size += nodes * case["topk"] * 4
            flops += 4 * DIM * rows * (per_node + tokens + 1)
        return {"bytes": size, "flops": flops}
    if case["op"] == "verify":
        # one row of the target (and of the draft) for each sequence's last node
        return {"bytes": case["batch"] * (case["vocab"] * 4 * (2 if case["draft"] else 1) + case["nodes"] * 16),
                "flops": case["batch"] * case["vocab"] * (3 if case["draft"] else 1)}
    width = case["gate_dim"] if case["gate_dim"] else case["dim"]
    rows = sum(1 + int(math.log2(n)) * 0.75 for n in _counts(dict(case, ragged=case["batch"] > 1)))
    return {"bytes": int(2 * rows * (2 * case["dim"] + 4 * width)) + 64 * case["batch"], "flops": 0}


# ------------------------------------------------------------------ exact values

def _exact_attend(s):
    """Node by node from the definition, in 64 bits."""
    ratio, slots = s["ratio"], s["slots"]
    cu, lens, parents = s["cu"].tolist(), s["lens"].tolist(), s["parents"].tolist()
    table, wtable = s["table"].long(), s["wtable"].long()
    flat, wflat = s["data"].reshape(-1, DIM), s["window"].reshape(-1, DIM)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    freq = torch.tensor([THETA ** (-2.0 * i / ROPE_DIM) for i in range(ROPE_DIM // 2)], dtype=torch.float64, device="cuda")

    def stored(b, first, last):
        j = torch.arange(first, last, device="cuda")
        return entry(b, j)

    def entry(b, j):
        where = table[b, torch.div(j, slots, rounding_mode="floor")] * slots + j % slots
        if s["scales"] is None:
            return flat[where].double()
        return flat[where].view(torch.float8_e4m3fn).double() * s["scales"].reshape(-1)[where].double()[:, None]

    for b, length in enumerate(lens):
        whole = None
        for i in range(cu[b + 1] - cu[b]):
            node = cu[b] + i
            family, a = [], i
            while a >= 0:
                family.append(a)
                a = parents[cu[b] + a]
            position = length + len(family) - 1
            begin = max(0, position + 1 - WINDOW)
            if s["topk"] is not None:
                j = s["topk"][node].long()
                values = entry(b, j[j >= 0])
            else:
                if whole is None:
                    whole = stored(b, 0, max(0, length + s["max_nodes"] - WINDOW) // ratio)
                values = whole[:begin // ratio]
            t = torch.arange(min(begin, length), length, device="cuda")
            window = wflat[wtable[b, t // BLOCK] * BLOCK + t % BLOCK].double() if t.numel() else wflat[:0].double()
            own_rows = s["k_tree"][[cu[b] + a for a in family]].double()
            v = torch.cat([values, window, own_rows])
            w = torch.softmax(s["q"][node].double() @ v.t() / math.sqrt(DIM), -1)
            o = w @ v
            z = torch.complex(o[:, ROPE_OFFSET::2].contiguous(), o[:, ROPE_OFFSET + 1::2].contiguous())
            z = z * torch.polar(torch.ones_like(freq), -position * freq)
            o[:, ROPE_OFFSET:] = torch.view_as_real(z).reshape(o.shape[0], ROPE_DIM)
            out[node] = o
    return out


def _exact_verify(s):
    """Sequence by sequence, child by child."""
    cu, parents, tokens = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    accept, sample = s["accept"].double().tolist(), s["sample"].double().tolist()
    batch = len(cu) - 1
    path = torch.full((batch, s["max_nodes"]), -1, dtype=torch.int32, device="cuda")
    length, following = [], []
    for b in range(batch):
        node, taken, going = 0, [0], True
        while going:
            going = False
            p = s["target"][cu[b] + node].double()
            rest, total = p.clone(), 1.0
            for child in range(node + 1, cu[b + 1] - cu[b]):
                if parents[cu[b] + child] != node:
                    continue
                x = tokens[cu[b] + child]
                chance = float(s["draft"][cu[b] + node, x]) if s["draft"] is not None else 1.0
                if accept[cu[b] + child] * chance * total < float(rest[x]):
                    node, going = child, True
                    taken.append(child)
                    break
                if s["draft"] is not None:
                    rest = torch.relu(rest - total * s["draft"][cu[b] + node].double())
                    total = float(rest.sum())
                else:
                    total -= float(rest[x])
                    rest[x] = 0.0
        if float(rest.sum()) <= 0:
            rest = p
        sums = torch.cumsum(rest, 0)
        over = torch.nonzero(sums > sample[b] * sums[-1])
        following.append(int(over[0]) if over.numel() else int(torch.nonzero(rest > 0)[-1]))
        path[b, :len(taken)] = torch.tensor(taken, dtype=torch.int32, device="cuda")
        length.append(len(taken))
    return {"path": path, "n_path": _int(length), "next": _int(following)}


def _exact_gather(s):
    """Row by row."""
    cu, path, n = s["cu"].tolist(), s["path"].tolist(), s["n_path"].tolist()
    x, gate, ends = torch.zeros_like(s["x"], dtype=torch.float64), torch.zeros_like(s["gate"], dtype=torch.float64), [0]
    for b, count in enumerate(n):
        rows = torch.tensor([cu[b] + i for i in path[b][:count]], device="cuda")
        x[ends[-1]:ends[-1] + count] = s["x"][rows].double()
        gate[ends[-1]:ends[-1] + count] = s["gate"][rows].double()
        ends.append(ends[-1] + count)
    return {"x": x, "gate": gate, "cu": _int(ends)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "verify": _exact_verify, "gather": _exact_gather}[case["op"]](s)
