"""The operators around the latent cache that are measured, in plain torch form.

Two families share one cache of rows [c^KV | k^R]:

* a tree of drafted tokens behind each sequence (speculative decoding):
  "tree_cache" writes the drafted rows and then keeps the accepted path,
  "tree_attn" verifies the tree in one pass of attention;
* attention over selected blocks of 64 cached tokens (long contexts):
  "block_scores" summarises blocks and scores them, "block_select" takes the
  best, "sparse_attn" attends the blocks that were taken.

`own = False` computes them with elementary torch operations in float32,
`own = True` through the library's entry points.
"""

import math

import torch

own = False

BLOCK = 64          # tokens per block of the selection, and per page
ROPE_BASE = 10000.0

V2 = dict(n_h=128, d_h=128, d_c=512, d_r=64, d_model=5120, dtype="bf16")
LITE = dict(n_h=16, d_h=128, d_c=512, d_r=64, d_model=2048, dtype="bf16")
TINY = dict(n_h=4, d_h=32, d_c=128, d_r=16, d_model=256, dtype="fp32")


def listed():
    return [
        # one user's chat with a small model, eight drafted tokens: latency
        dict(name="tree_attn_lite_b1", op="tree_attn", **LITE, B=1, T=8, lo=500, hi=500, page=0),
        # the ordinary serving batch, a tree of eight
        dict(name="tree_attn_v2_b16", op="tree_attn", **V2, B=16, T=8, lo=8192, hi=8192, page=0),
        # mixed lengths in a paged pool, an odd tree
        dict(name="tree_attn_lite_paged", op="tree_attn", **LITE, B=32, T=13, lo=256, hi=32768, page=64),
        # the largest tree, over documents
        dict(name="tree_attn_v2_t64", op="tree_attn", **V2, B=2, T=64, lo=12000, hi=16384, page=64),
        # a small float32 model
        dict(name="tree_cache_tiny", op="tree_cache", **TINY, B=2, T=5, lo=17, hi=64, page=0),
        # the cache side of a drafted step of a large batch
        dict(name="tree_cache_v2_b64", op="tree_cache", **V2, B=64, T=16, lo=200, hi=1000, page=64),
        # four long documents right after their prompt: every block is summarised
        dict(name="block_scores_lite_prompt", op="block_scores", **LITE, B=4, lo=131072, hi=131072, new=131072, page=0),
        # one decode step of the serving batch: one block per sequence changes
        dict(name="block_scores_v2_step", op="block_scores", **V2, B=64, lo=8000, hi=8192, new=1, page=64),
        # one long document
        dict(name="block_select_b1", op="block_select", B=1, lo=131000, hi=131000, k=64, first=1, last=2),
        # many sequences of mixed lengths
        dict(name="block_select_b128", op="block_select", B=128, lo=256, hi=32768, k=32, first=1, last=1),
        # the serving batch with 2048 of its 8192 tokens attended
        dict(name="sparse_attn_v2_b64", op="sparse_attn", **V2, B=64, lo=8000, hi=8192, k=32, page=0),
        # four long documents with 4096 of their tokens attended
        dict(name="sparse_attn_lite_b4", op="sparse_attn", **LITE, B=4, lo=131072, hi=131072, k=64, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree_attn", "tree_cache", "block_scores", "block_select", "sparse_attn"])
    shape = dict(rng.choice([V2, LITE, LITE, TINY]))
    if shape["n_h"] == 16 and rng.random() < 0.4:
        shape["n_h"] = 32
    page = rng.choice([0, 64])
    tiny, heads = shape["dtype"] == "fp32", shape["n_h"]
    if op == "block_select":
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 64, min(131072, 1048576 // B))
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, k=_log_int(rng, 4, 128), first=rng.randint(0, 2),
                    last=rng.randint(1, 3))
    if op == "tree_cache":
        T = _log_int(rng, 1, 64)
        B = _log_int(rng, 1, max(1, min(64, 1024 // T)))
        hi = _log_int(rng, 20, 1000)
        return dict(op=op, **shape, B=B, T=T, lo=rng.randint(1, hi), hi=hi, page=page)
    if op == "tree_attn":
        T = _log_int(rng, 1, 64)
        B = _log_int(rng, 1, 4 if tiny else 64)
        # tokens x query rows at most those of the largest listed case
        most = 300 if tiny else max(64, min(32768, 200_000_000 // (B * T * heads)))
        hi = _log_int(rng, 16, most)
        return dict(op=op, **shape, B=B, T=T, lo=rng.randint(1, hi), hi=hi, page=page)
    B = _log_int(rng, 1, 8 if tiny else 64)
    hi = _log_int(rng, 64, 2000 if tiny else min(131072, 524288 // B))
    lo = rng.randint(1, hi)
    if op == "block_scores":
        return dict(op=op, **shape, B=B, lo=lo, hi=hi, new=rng.choice([1, rng.randint(1, lo), lo]), page=page)
    return dict(op=op, **shape, B=B, lo=lo, hi=hi, k=min(_log_int(rng, 4, 128), 2048 // B), page=page)


def _lengths(case):
    """Cached tokens of each sequence, from lo to hi (evenly in the logarithm), in a mixed order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    step = next(s for s in (7, 5, 3, 2, 1) if math.gcd(s, B) == 1)
    return [int(round(lo * (hi / lo) ** ((b * step % B) / max(1, B - 1)))) for b in range(B)]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)

    def normal(*size, std=1.0):
        return (torch.randn(*size, generator=g, device=dev) * std).to(_dtype(case))

    def uniform(*size):
        return torch.rand(*size, generator=g, device=dev)

    B, op = case["B"], case["op"]
    lens = _lengths(case)
    s = dict(case)
    s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    T = case.get("T", 0)
    longest = max(lens) + T
    blocks = -(-longest // BLOCK)
    if op == "block_select":
        # scores as a softmax leaves them: most of the mass in few blocks, equal values among the rest
        mass = torch.exp(3.0 * torch.randn(B, blocks, generator=g, device=dev))
        mass = torch.where(uniform(B, blocks) < 0.1, torch.floor(mass), mass)
        s["scores"] = mass / mass.sum(1, keepdim=True)
        s["sel"] = torch.empty(B, case["k"], dtype=torch.int32, device=dev)
        s["n_sel"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["n_blocks"] = blocks
        return s

    n_h, d_c, d_r, d_model = (case[k] for k in ("n_h", "d_c", "d_r", "d_model"))
    D = d_c + d_r
    s["D"], s["scale"] = D, 1.0 / math.sqrt(case["d_h"] + d_r)
    if case["page"]:
        # a pool with room to spare, the pages of each sequence anywhere in it
        pool = B * blocks + 3
        s["cache"] = normal(pool, BLOCK, D)
        s["table"] = torch.randperm(pool, generator=g, device=dev)[: B * blocks].reshape(B, blocks).to(torch.int32)
        s["cache_len"], s["max_blk"] = pool, blocks
    else:
        s["cache_len"], s["max_blk"], s["table"] = longest, 0, None
        s["cache"] = normal(B, longest, D)

    if T:
        # a random tree: each drafted token hangs below an earlier one or the last cached token
        parent = [-1] * T
        pick = torch.rand(T, generator=torch.Generator().manual_seed(seed)).tolist()
        bits, depth = [0] * T, [0] * T
        for t in range(T):
            parent[t] = int(pick[t] * (t + 1)) - 1
            up = parent[t]
            bits[t] = (bits[up] if up >= 0 else 0) | (1 << t)
            depth[t] = depth[up] + 1 if up >= 0 else 0
        signed = [b - (1 << 64) if b >> 63 else b for b in bits]
        s["mask"] = torch.tensor(signed, dtype=torch.int64, device=dev).repeat(B, 1)
        s["depth"] = torch.tensor(depth, dtype=torch.int32, device=dev).repeat(B, 1)
        # the accepted path: the deepest token's, cut at another depth for each sequence
        deepest = max(range(T), key=lambda t: depth[t])
        path = [t for t in range(T) if bits[deepest] >> t & 1]
        s["path"] = torch.tensor(path + [0] * (T - len(path)), dtype=torch.int32, device=dev).repeat(B, 1)
        s["n_path"] = torch.tensor([(b * 3 + 1) % (len(path) + 1) for b in range(B)], dtype=torch.int32, device=dev)
    if op == "tree_cache":
        s["h"] = normal(B, T, d_model)
        s["w_dkv"] = normal(d_c, d_model, std=d_model ** -0.5)
        s["w_kr"] = normal(d_r, d_model, std=d_model ** -0.5)
        s["new_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        return s

    # absorbed queries: W_UK^T q over d_c columns, and a rotated part of unit variance
    q_shape = (B, T, n_h) if T else (B, n_h)
    s["q"] = torch.cat([normal(*q_shape, d_c, std=math.sqrt(case["d_h"] / d_c)), normal(*q_shape, d_r)], -1)
    s["out"] = torch.empty(*q_shape, d_c, dtype=_dtype(case), device=dev)
    s["lse"] = torch.empty(*q_shape, dtype=torch.float32, device=dev)
    if op == "block_scores":
        s["begin"] = (s["ctx"] - case["new"]).clamp(min=0)
        s["key_blocks"] = blocks
        s["keys"] = _block_means(s, torch.float32)[0]
        s["scores"] = torch.empty(B, blocks, dtype=torch.float32, device=dev)
    if op == "sparse_attn":
        # blocks taken at random, the first and the last of each sequence among them
        n_blk = (s["ctx"] + BLOCK - 1) // BLOCK
        at = torch.arange(blocks, device=dev)
        order = uniform(B, blocks)
        order = torch.where((at == 0) | (at == n_blk[:, None] - 1), 2.0, order)
        order = torch.where(at < n_blk[:, None], order, -1.0)
        k = case["k"]
        if k > blocks:
            order = torch.nn.functional.pad(order, (0, k - blocks), value=-1.0)
        top = torch.sort(order, 1, descending=True)
        s["n_sel"] = n_blk.clamp(max=k).to(torch.int32)
        idx = torch.where(top.values[:, :k] >= 0, top.indices[:, :k], 1 << 30).sort(1).values
        s["sel"] = torch.where(idx < 1 << 30, idx, -1).to(torch.int32)
    return s


# --------------------------------------------------------------- plain forms


def _rows(s, n):
    """The first n cached rows of every sequence, float32 [B, n, D]."""
    if s["page"]:
        rows = s["cache"][s["table"][:, : -(-n // BLOCK)].long()].reshape(s["B"], -1, s["D"])
    else:
        rows = s["cache"]
    return rows[:, :n].float()


def _attend(q, rows, allowed, scale, d_c, dtype):
    """Softmax attention of q [B, R, D] over rows [B, L, D] where allowed
    [B, R or 1, L]; a query that may attend nothing gets zeros and -inf."""
    x = torch.bmm(q.float(), rows.transpose(1, 2)) * scale
    x = x.masked_fill(~allowed, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p, rows[..., :d_c]) / torch.where(total > 0, total, 1.0)
    return out.to(dtype), (m + torch.log(total)).squeeze(-1)


def _tree_attn(s):
    B, T, n_h = s["B"], s["T"], s["n_h"]
    n = max(_lengths(s)) + T
    at = torch.arange(n, device="cuda")
    ctx = s["ctx"].long()[:, None, None]
    slot = (at - ctx).clamp(0, T - 1).expand(B, T, n)          # drafted slot of each column
    bit = (s["mask"][:, :, None] >> slot) & 1
    allowed = (at < ctx) | ((at < ctx + T) & (bit == 1))
    allowed = allowed[:, :, None].expand(B, T, n_h, n).reshape(B, T * n_h, n)
    out, lse = _attend(s["q"].reshape(B, T * n_h, -1), _rows(s, n), allowed, s["scale"], s["d_c"], s["q"].dtype)
    return out.reshape(B, T, n_h, -1), lse.reshape(B, T, n_h)


def _flat_rows(s, pos):
    """Row numbers in the flattened cache of positions pos [B, n]."""
    if s["page"]:
        return s["table"].long().gather(1, pos // BLOCK) * BLOCK + pos % BLOCK
    return torch.arange(s["B"], device="cuda")[:, None] * s["cache_len"] + pos


def _rope(x, pos, d_r):
    theta = ROPE_BASE ** (-2.0 * torch.arange(d_r // 2, dtype=torch.float64, device="cuda") / d_r)
    angle = pos.double()[..., None] * theta
    co, si = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * co - x1 * si, x0 * si + x1 * co], -1).flatten(-2)


def _tree_cache(s):
    B, T = s["B"], s["T"]
    ctx = s["ctx"].long()[:, None]
    flat = s["cache"].view(-1, s["D"])
    c = s["h"].float() @ s["w_dkv"].float().T
    r = _rope(s["h"].float() @ s["w_kr"].float().T, ctx + s["depth"], s["d_r"])
    t = torch.arange(T, device="cuda")
    flat[_flat_rows(s, ctx + t)] = torch.cat([c, r], -1).to(flat.dtype)
    # the accepted rows move to the front; the slots after them keep what they hold
    source = torch.where(t < s["n_path"][:, None], s["path"], t).long()
    flat[_flat_rows(s, ctx + t)] = flat[_flat_rows(s, ctx + source)]
    return s["cache"], s["ctx"] + s["n_path"]


def _block_means(s, dtype):
    """Mean row of every block [B, blocks, D] over its cached tokens, and their number."""
    blocks = -(-max(_lengths(s)) // BLOCK)
    at = torch.arange(blocks * BLOCK, device="cuda")
    rows = torch.nn.functional.pad(_rows(s, max(_lengths(s))), (0, 0, 0, blocks * BLOCK - max(_lengths(s))))
    here = at < s["ctx"][:, None]
    rows = torch.where(here[..., None], rows, 0.0).reshape(s["B"], blocks, BLOCK, -1)
    n = here.reshape(s["B"], blocks, BLOCK).sum(-1)
    means = rows.to(dtype).sum(2) / n.clamp(min=1)[..., None]
    return means.to(s["cache"].dtype) if dtype == torch.float32 else means, n


def _block_scores(s):
    B, blocks = s["B"], s["key_blocks"]
    # blocks that hold new tokens are summarised again
    changed = min(blocks, (s["new"] + BLOCK - 2) // BLOCK + 1)
    j = s["begin"].long()[:, None] // BLOCK + torch.arange(changed, device="cuda")
    pos = j[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    here = pos < s["ctx"][:, None, None]
    rows = s["cache"].view(-1, s["D"])[_flat_rows(s, pos.clamp(max=max(_lengths(s)) - 1).reshape(B, -1))]
    rows = torch.where(here.reshape(B, -1, 1), rows.float(), 0.0).reshape(B, changed, BLOCK, -1)
    means = rows.sum(2) / here.sum(-1).clamp(min=1)[..., None]
    place = j % blocks
    old = s["keys"].gather(1, place[..., None].expand(B, changed, s["D"]))
    means = torch.where(here[:, :, :1], means.to(old.dtype), old)
    s["keys"].scatter_(1, place[..., None].expand(B, changed, s["D"]), means)
    # every head spreads its attention over the blocks by their mean rows; the heads' shares are added
    n = (s["ctx"][:, None] - BLOCK * torch.arange(blocks, device="cuda")).clamp(0, BLOCK)
    x = torch.bmm(s["q"].float(), s["keys"].float().transpose(1, 2)) * s["scale"]
    x = x + torch.log(n.float())[:, None]
    x = x.masked_fill((n == 0)[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return s["keys"], (p / torch.where(total > 0, total, 1.0)).sum(1)


def _block_select(s):
    blocks, k = s["n_blocks"], s["k"]
    at = torch.arange(blocks, device="cuda")
    n_blk = ((s["ctx"] + BLOCK - 1) // BLOCK)[:, None]
    x = torch.where((at < s["first"]) | (at >= n_blk - s["last"]), math.inf, s["scores"])
    x = x.masked_fill(at >= n_blk, -math.inf)
    best = torch.sort(x, dim=1, descending=True, stable=True).indices
    if k > blocks:
        best = torch.nn.functional.pad(best, (0, k - blocks))
    n_sel = n_blk.clamp(max=k)
    best = torch.where(torch.arange(k, device="cuda") < n_sel, best[:, :k], blocks).sort(1).values
    return torch.where(best < blocks, best, -1).to(torch.int32), n_sel[:, 0].to(torch.int32)


def _selected(s):
    """Positions [B, k * 64] of the tokens of the taken blocks, and which of them exist."""
    sel = s["sel"].long()
    pos = (sel.clamp(min=0)[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(s["B"], -1)
    here = (pos < s["ctx"][:, None]) & (sel >= 0).repeat_interleave(BLOCK, 1)
    return torch.where(here, pos, 0), here


def _sparse_attn(s):
    pos, here = _selected(s)
    rows = s["cache"].view(-1, s["D"])[_flat_rows(s, pos)].float()
    return _attend(s["q"], rows, here[:, None], s["scale"], s["d_c"], s["q"].dtype)


# ------------------------------------------------------- the library's calls

_handles = {}


def _handle(s):
    """The program's handle for a model's configuration."""
    import head_latent_attention_09_b200 as M
    key = tuple(s.get(k, 0) for k in ("n_h", "d_h", "d_c", "d_r", "d_model", "page", "dtype"))
    if key not in _handles:
        if s["op"] == "block_select":
            cfg = M.mla_config(n_h=16, d_h=128, d_c=512, d_r=64, d_model=2048, page_size=0, rope_base=ROPE_BASE,
                               dtype=M.MLA_BF16)
        else:
            cfg = M.mla_config(n_h=s["n_h"], d_h=s["d_h"], d_c=s["d_c"], d_r=s["d_r"], d_model=s["d_model"],
                               page_size=s["page"], rope_base=ROPE_BASE,
                               dtype=M.MLA_BF16 if s["dtype"] == "bf16" else M.MLA_FP32)
        _handles[key] = M.mla_create(cfg)
    return M, _handles[key]


def _workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.empty(max(256, size()), dtype=torch.uint8, device="cuda")
    return s["ws"], s["ws"].numel()


def _own_tree_attn(s):
    M, h = _handle(s)
    ws, size = _workspace(s, lambda: M.mla_tree_workspace_size(h, s["B"], s["T"], 0))
    M.mla_tree_attn(h, s["q"], s["cache"], s["cache_len"], s["table"], s["max_blk"], s["ctx"], s["mask"], s["B"],
                    s["T"], 0, s["out"], s["lse"], ws, size)
    return s["out"], s["lse"]


def _own_tree_cache(s):
    M, h = _handle(s)
    M.mla_cache_append_tree(h, s["h"], s["B"], s["T"], s["ctx"], s["depth"], s["w_dkv"], s["w_kr"], s["cache"],
                            s["cache_len"], s["table"], s["max_blk"])
    M.mla_tree_accept(h, s["cache"], s["cache_len"], s["table"], s["max_blk"], s["ctx"], s["path"], s["n_path"],
                      s["B"], s["T"], s["new_len"])
    return s["cache"], s["new_len"]


def _own_block_scores(s):
    M, h = _handle(s)
    ws, size = _workspace(s, lambda: M.mla_block_scores_workspace_size(h, s["B"], s["key_blocks"]))
    M.mla_block_keys(h, s["cache"], s["cache_len"], s["table"], s["max_blk"], s["begin"], s["ctx"], s["B"], s["new"],
                     s["keys"], s["key_blocks"])
    M.mla_block_scores(h, s["q"], s["keys"], s["key_blocks"], s["ctx"], s["B"], s["scores"], ws, size)
    return s["keys"], s["scores"]


def _own_block_select(s):
    M, h = _handle(s)
    M.mla_block_select(h, s["scores"], s["n_blocks"], s["ctx"], s["B"], s["k"], s["first"], s["last"], s["sel"],
                       s["n_sel"])
    return s["sel"], s["n_sel"]


def _own_sparse_attn(s):
    M, h = _handle(s)
    ws, size = _workspace(s, lambda: M.mla_decode_workspace_size(h, s["B"], 0))
    M.mla_decode_attn_sparse(h, s["q"], s["cache"], s["cache_len"], s["table"], s["max_blk"], s["ctx"], s["sel"],
                             s["n_sel"], s["k"], s["B"], 0, ws, size)
    M.mla_combine_splits(h, ws, size, s["B"], 0, s["out"], s["lse"])
    return s["out"], s["lse"]


def run(state):
    op = state["op"]
    if own:
        if op == "tree_attn":
            return _own_tree_attn(state)
        if op == "tree_cache":
            return _own_tree_cache(state)
        if op == "block_scores":
            return _own_block_scores(state)
        if op == "block_select":
            return _own_block_select(state)
        return _own_sparse_attn(state)
    if op == "tree_attn":
        return _tree_attn(state)
    if op == "tree_cache":
        return _tree_cache(state)
    if op == "block_scores":
        return _block_scores(state)
    if op == "block_select":
        return _block_select(state)
    return _sparse_attn(state)


# ---------------------------------------------------------- work and oracle


def work(case):
    B, op = case["B"], case["op"]
    lens = _lengths(case)
    blocks = [-(-n // BLOCK) for n in lens]
    if op == "block_select":
        return {"bytes": 4 * sum(blocks) + 4 * B * (case["k"] + 2), "flops": 2 * sum(blocks)}
    e = 2 if case["dtype"] == "bf16" else 4
    n_h, d_c, d_model = case["n_h"], case["d_c"], case["d_model"]
    D, T = d_c + case["d_r"], case.get("T", 1)
    q, out = n_h * D * e, n_h * (d_c * e + 4)
    if op == "tree_attn":
        return {"bytes": sum(lens) * D * e + B * T * (D * e + q + out + 8) + 4 * B,
                "flops": 2 * n_h * (D + d_c) * T * (sum(lens) + B)}
    if op == "tree_cache":
        return {"bytes": D * d_model * e + B * T * (d_model + D) * e + 8 * B * T + 12 * B,
                "flops": 2 * B * T * D * d_model}
    if op == "block_scores":
        new = sum(min(n, -(-case["new"] // BLOCK) * BLOCK) for n in lens)
        return {"bytes": new * D * e + sum(blocks) * (D * e + 4) + B * (q + 8),
                "flops": 2 * n_h * D * sum(blocks) + new * D}
    taken = sum(min(n, case["k"] * BLOCK) for n in lens)
    return {"bytes": taken * D * e + B * (q + out + 4 * case["k"] + 8), "flops": 2 * n_h * (D + d_c) * taken}


def _exact_rows(s, b, pos):
    """Cached rows of sequence b at the listed positions, float64."""
    if s["page"]:
        page = s["table"][b].long()[torch.div(pos, BLOCK, rounding_mode="floor")]
        return s["cache"][page, pos % BLOCK].double()
    return s["cache"][b, pos].double()


def _exact_softmax(q, rows, may, s):
    """One head's or one token's softmax attention, with the log of its sum."""
    score = (q @ rows.T) * s["scale"]
    score = torch.where(may, score, torch.full_like(score, -math.inf))
    lse = torch.logsumexp(score, -1)
    p = torch.exp(score - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return p @ rows[:, : s["d_c"]], lse


def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    lens = _lengths(case)
    if op == "block_select":
        return None      # whole numbers, which the plain form has exactly
    if op == "tree_attn":
        T, out, lse = case["T"], s["q"].new_empty(s["out"].shape, dtype=torch.float64), s["lse"].double()
        words = s["mask"].tolist()
        for b, n in enumerate(lens):
            rows = _exact_rows(s, b, torch.arange(n + T, device="cuda"))
            for t in range(T):
                may = torch.ones(n + T, dtype=torch.bool)
                may[n:] = torch.tensor([words[b][t] >> u & 1 == 1 for u in range(T)])
                out[b, t], lse[b, t] = _exact_softmax(s["q"][b, t].double(), rows, may.cuda(), s)
        return out, lse
    if op == "tree_cache":
        T, cache = case["T"], s["cache"].double()
        w = torch.cat([s["w_dkv"], s["w_kr"]]).double()
        freq = [ROPE_BASE ** (-2.0 * i / case["d_r"]) for i in range(case["d_r"] // 2)]
        freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            new = s["h"][b].double() @ w.T
            turn = torch.polar(torch.ones_like(freq), (n + s["depth"][b].double())[:, None] * freq)
            pair = torch.view_as_complex(new[:, case["d_c"]:].reshape(T, -1, 2).contiguous())
            new[:, case["d_c"]:] = torch.view_as_real(pair * turn).reshape(T, -1)
            kept = s["path"][b, : int(s["n_path"][b])].long()
            new = torch.cat([new[kept], new[len(kept):]])
            for t in range(T):
                p = n + t
                if case["page"]:
                    cache[s["table"][b, p // BLOCK].long(), p % BLOCK] = new[t]
                else:
                    cache[b, p] = new[t]
        return cache, None
    if op == "block_scores":
        keys, scores = s["keys"].double(), torch.zeros_like(s["scores"], dtype=torch.float64)
        for b, n in enumerate(lens):
            j0, blocks = int(s["begin"][b]) // BLOCK, -(-n // BLOCK)
            rows = _exact_rows(s, b, torch.arange(j0 * BLOCK, n, device="cuda"))
            for j in range(j0, blocks):
                keys[b, j] = rows[(j - j0) * BLOCK: (j - j0 + 1) * BLOCK].mean(0)
            # the scores are those of the keys as they are kept
            kept = keys[b, :blocks].to(s["keys"].dtype).double()
            size = torch.full((blocks,), float(BLOCK), dtype=torch.float64, device="cuda")
            size[-1] = n - BLOCK * (blocks - 1)
            share = torch.softmax(s["q"][b].double() @ kept.T * s["scale"] + size.log(), -1)
            scores[b, :blocks] = share.sum(0)
        return keys, scores
    out, lse = s["q"].new_empty(s["out"].shape, dtype=torch.float64), s["lse"].double()
    for b, n in enumerate(lens):
        pos = [p for j in s["sel"][b].tolist() if j >= 0 for p in range(j * BLOCK, min(n, (j + 1) * BLOCK))]
        rows = _exact_rows(s, b, torch.tensor(pos, device="cuda"))
        may = torch.ones(len(pos), dtype=torch.bool, device="cuda")
        out[b], lse[b] = _exact_softmax(s["q"][b].double(), rows, may, s)
    return out, lse
