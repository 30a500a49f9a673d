"""Rotary positions and the paged bf16 KV cache as measured work: rope, paged_append,
paged_attn and paged_keep.

The cache holds bf16 pages [n_pages, Hkv, page, D] for keys and for values; position p of
sequence b is row p % page of page tables[b, p // page]. Four kinds of case:

  rope    queries and keys of T tokens normed per head (optional) and rotated by their
          positions, the first `rot` values of each head;
  append  new tokens' keys normed, rotated and written with their values into the pages at
          positions starts[b].. of each sequence; their queries normed and rotated alongside;
  attn    attention of each sequence's last news[b] tokens over its lens[b] cached positions:
          causal (one token a sequence is decode, many a prompt or a chunk of one), or a tree
          of drafts, each of which sees the context and its own ancestors;
  keep    the accepted path through a tree of drafts moved to the positions right after the
          context.

Tokens of all sequences are packed end to end. With `fused` the new tokens' q, k and v are
column ranges of one projection output, so tokens are strided. Pages lie in the pool in any
order; what the cases leave of it unused holds values too, and the tables say -1 there.
"""
import math
import random

import numpy as np
import torch

own = False

MODEL = dict(Hq=16, Hkv=2, D=256, page=64)  # the layer's head layout
EPS = 1e-6


def _csv(values):
    return ",".join(str(int(v)) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _turn(rot, layout="half", norm=True, scaling="plain", base=1e7, factor=1.0, orig=0, offset=0.0):
    """How a case norms and rotates its heads."""
    return dict(rot=rot, layout=layout, norm=norm, scaling=scaling, base=base, factor=factor, orig=orig, offset=offset)


def listed():
    batch8 = "4096,32768,1,17000,65536,8191,777,20000"
    return [
        # one decode step of 64 sequences, anywhere in a 128K context: a quarter of each head turns
        dict(name="rope-decode-b64", kind="rope", fused=True, seed=1, T=64, top=131072, **MODEL, **_turn(64)),
        # a chunk of a long document, whole heads turned pair by pair, positions scaled to a longer context
        dict(name="rope-long-8192", kind="rope", fused=True, seed=2, T=8192, top=1 << 20, Hq=40, Hkv=8, D=128, page=64,
             **_turn(128, "pairs", False, "ramp", 1e4, 32.0, 32768)),
        # one decode step of 64 sequences: each appends a token
        dict(name="append-decode-b64", kind="append", fused=True, tree=False, seed=3,
             lens=_csv(1 + (977 * i) % 1500 for i in range(64)), news=_csv([1] * 64), **MODEL, **_turn(64, offset=1.0)),
        # a prompt of 4096 tokens beside chunks that start and end inside pages, one of them empty
        dict(name="append-ragged", kind="append", fused=True, tree=False, seed=4, Hq=16, Hkv=4, D=128, page=32,
             lens="4096,777,4097,64,2049", news="4096,0,2097,1,516", **_turn(64, "pairs", True, "bands", 5e5, 8.0, 8192)),
        # decode over a short context: latency
        dict(name="attn-decode-300", kind="attn", fused=False, tree=False, seed=5, lens="300", news="1", **MODEL),
        # decode of a ragged batch
        dict(name="attn-decode-batch8", kind="attn", fused=True, tree=False, seed=6, lens=batch8, news=_csv([1] * 8),
             **MODEL),
        # a small tree of drafts of each of 16 sequences verified at once; 4 query heads a KV head
        dict(name="attn-tree-b16", kind="attn", fused=True, tree=True, seed=7, Hq=16, Hkv=4, D=128, page=16,
             lens=_csv(700 + 491 * i for i in range(16)), news=_csv(3 + 4 * i % 29 for i in range(16))),
        # wide trees of two sequences with long contexts
        dict(name="attn-tree-wide", kind="attn", fused=False, tree=True, seed=8, lens="20000,9001", news="200,77", **MODEL),
        # a whole prompt
        dict(name="attn-prompt-4096", kind="attn", fused=True, tree=False, seed=9, lens="4096", news="4096", **MODEL),
        # a 2048-token chunk of a long prompt over what is cached already
        dict(name="attn-chunk-2048-of-18k", kind="attn", fused=False, tree=False, seed=10, lens="18432", news="2048",
             **MODEL),
        # the accepted drafts of 64 sequences
        dict(name="keep-b64", kind="keep", seed=11, lens=_csv(100 + (331 * i) % 1500 for i in range(64)),
             news=_csv([32] * 64), kept=_csv(i % 9 for i in range(64)), **MODEL),
        # long paths of many sequences, small pages
        dict(name="keep-wide", kind="keep", seed=12, Hq=8, Hkv=8, D=128, page=16, lens=_csv([700 + i for i in range(200)]),
             news=_csv([200] * 200), kept=_csv([20 + i % 21 for i in range(200)])),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _any_turn(rng, D):
    rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128, 256) if r <= D] + [D])
    scaling = rng.choice(["plain", "linear", "bands", "ramp"])
    return _turn(rot, rng.choice(["half", "pairs"]), rng.random() < 0.6, scaling, rng.choice([1e4, 5e5, 1e6, 1e7]),
                 1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0, 32.0]), rng.choice([4096, 8192, 32768]),
                 rng.choice([0.0, 1.0]))


def draw(rng):
    kind = rng.choice(["rope", "append", "attn", "attn", "attn", "keep"])
    Hq, Hkv, D = rng.choice([(16, 2, 256), (16, 2, 256), (8, 8, 128), (4, 1, 64), (6, 3, 256), (16, 4, 128), (40, 8, 128)])
    c = dict(kind=kind, seed=rng.randrange(1 << 20), Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]))
    if kind != "keep":
        c.update(fused=rng.random() < 0.5)
    if kind == "rope":
        c.update(T=_log(rng, 1, (1 << 25) // ((Hq + Hkv) * D)), top=_log(rng, 64, 1 << 20), **_any_turn(rng, D))
        return c
    B = _log(rng, 1, 24)
    rows = (1 << 26) // (Hkv * D)  # positions of the largest cache: 131072 of 2 heads of 256
    lens = [min(_log(rng, 1, rows // 2), rows // B) for _ in range(B)]
    if kind == "append":  # bounded by the largest listed one
        most = (1 << 24) // ((Hq + 2 * Hkv) * D * B)
        form = rng.choice(["one", "tree", "many"])
        news = [1 if form == "one" else min(n, rng.randint(0, 63 if form == "tree" else most), most) for n in lens]
        c.update(tree=form == "tree", **_any_turn(rng, D))
    elif kind == "attn":
        form = rng.choice(["one", "tree", "tree", "many"])
        news = [1] * B
        if form == "tree":
            wide = rng.choice([8, 64, 256])
            news = [min(n, rng.randint(0, wide)) for n in lens]
        elif form == "many":
            news = [rng.randint(0, n) for n in lens]
            if rng.random() < 0.3:
                news = list(lens)
        most = (1 << 29) // (Hq * B * max(lens))  # the padded scores stay within the largest listed ones
        news = [min(n, max(1, most)) for n in news]
        c.update(tree=form == "tree")
    else:
        news = [min(n, rng.randint(1, 256)) for n in lens]
        c.update(kept=_csv(rng.randint(0, min(n, 40)) for n in news))
    if sum(news) == 0:
        news[0] = 1
    c.update(lens=_csv(lens), news=_csv(news))
    return c


# ------------------------------------------------------------------ inputs ---

def _parents(rng, n):
    """The parent of each of n drafts, which come after their parents; the first one's is the context."""
    return [-1] + [rng.randint(max(0, i - 9), i - 1) for i in range(1, n)]


def _path(rng, n, kept):
    """`kept` drafts of n in increasing order, each at its place already or behind all places."""
    head = rng.randint(0, kept)
    tail = sorted(rng.sample(range(kept, n), min(kept - head, n - kept)))
    return (list(range(kept - len(tail))) + tail)


def _frequencies(case):
    """The angle per position of every pair, in radians (fp64), and the factor on cosine and sine."""
    rot, base, f, orig = case["rot"], case["base"], case["factor"], case["orig"]
    w = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "bands":  # long waves stretched, short ones kept, in between a mixture
        turns = orig * w / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return w * keep + w / f * (1 - keep), 1.0
    if case["scaling"] == "ramp":  # a ramp over the pairs between 32 turns and 1 turn in the original context
        def at(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0
    return w, 1.0


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed((seed * 1_000_003 + case["seed"]) % (1 << 62))
    rng = random.Random(seed * 7919 + case["seed"])
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    st = dict(case=case, dev=dev)
    # keys vary in size from channel to channel
    gain = torch.exp(0.4 * normal(Hkv * D))
    if case["kind"] == "rope":
        T = case["T"]
        first = rng.randrange(max(1, case["top"] - T))
        pos = [first + i for i in range(T)] if T > 1000 else [rng.randrange(case["top"]) for _ in range(T)]
        st["positions"] = ints(pos)
    else:
        lens, news = _ints(case["lens"]), _ints(case["news"])
        B, T = len(lens), sum(news)
        starts = [n - m for n, m in zip(lens, news)]
        need = [-(-n // page) for n in lens]
        P, n_pages = max(need), sum(need) + 3
        where = torch.randperm(n_pages, generator=gen, device=dev).int()
        tables = torch.full((B, P), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, k in enumerate(need):
            tables[b, :k] = where[at:at + k]
            at += k
        st.update(B=B, L=max(lens), P=P, n_pages=n_pages, tables=tables, nmax=max(news), lens=ints(lens),
                  starts=ints(starts), offsets=ints(np.concatenate([[0], np.cumsum(news)]).tolist()))
        st["k_pages"] = (normal(n_pages, Hkv, page, D) * gain.view(1, Hkv, 1, D)).to(torch.bfloat16)
        st["v_pages"] = normal(n_pages, Hkv, page, D).to(torch.bfloat16)
        if case["kind"] == "keep":
            kept = _ints(case["kept"])
            path = np.zeros((B, max(max(kept), 1)), dtype=np.int32)
            for b, (n, k) in enumerate(zip(news, kept)):
                path[b, :k] = _path(rng, n, k)
            st.update(kept=ints(kept), path=torch.from_numpy(path).to(dev))
            T = 0
        elif case["tree"]:
            words = max(1, -(-max(news) // 64))
            seen = np.zeros((T, words), dtype=np.uint64)
            pos, t = [], 0
            for s, n in zip(starts, news):
                for i, parent in enumerate(_parents(rng, n) if n else []):
                    if parent >= 0:
                        seen[t] = seen[t - i + parent]
                    seen[t, i // 64] |= np.uint64(1 << (i % 64))
                    pos.append(s if parent < 0 else pos[t - i + parent] + 1)
                    t += 1
            st.update(words=words, tree=torch.from_numpy(seen.view(np.int64)).to(dev), positions=ints(pos))
    st["T"] = T
    st["qs"] = st["kvs"] = 0
    if T and case["fused"]:  # one projection output [T, (Hq + 2 Hkv) D]
        w = (Hq + 2 * Hkv) * D
        x = normal(T, w)
        x[:, Hq * D:(Hq + Hkv) * D] *= gain
        x = x.to(torch.bfloat16)
        st["q"] = x[:, :Hq * D].view(T, Hq, D)
        st["kn"] = x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        st["vn"] = x[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        st["qs"] = st["kvs"] = w
    elif T:
        st["q"] = normal(T, Hq, D).to(torch.bfloat16)
        if case["kind"] != "attn":
            st["kn"] = (normal(T, Hkv, D) * gain.view(1, Hkv, D)).to(torch.bfloat16)
            st["vn"] = normal(T, Hkv, D).to(torch.bfloat16)
    if "rot" in case:
        w, magnitude = _frequencies(case)
        st.update(w=w.to(dev), magnitude=magnitude, q_gain=None, k_gain=None)
        if case["norm"]:
            st["q_gain"] = (1 - case["offset"] + 0.2 * normal(D)).to(torch.bfloat16)
            st["k_gain"] = (1 - case["offset"] + 0.2 * normal(D)).to(torch.bfloat16)
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a serving loop keeps between calls: shapes, the rotation's table, output buffers, the workspace."""
    import bit_grouped_expert_moe_gb300 as m
    c, dev, T = st["case"], st["dev"], st["T"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    st["m"] = m
    if "rot" in c:
        kinds = dict(plain=m.ROPE_PLAIN, linear=m.ROPE_LINEAR, bands=m.ROPE_BANDS, ramp=m.ROPE_RAMP)
        table = m.rope_table(c["rot"], base=c["base"], scaling=kinds[c["scaling"]], factor=c["factor"],
                             original=c["orig"], device=dev)
        st["spec"] = m.rope_spec(table, layout=m.ROPE_HALF if c["layout"] == "half" else m.ROPE_PAIRS,
                                 norm=m.ROPE_NORM_QK if c["norm"] else 0, q_gain=st["q_gain"], k_gain=st["k_gain"],
                                 eps=EPS, gain_offset=c["offset"])
    if c["kind"] != "rope":
        st["cache"] = m.PagedCache(st["k_pages"], st["v_pages"], st["tables"])
        st["shape"] = m.paged_shape(st["B"], T, Hq, Hkv, D, c["page"], st["n_pages"], st["P"],
                                    tree_words=st["words"] if c["kind"] == "attn" and c["tree"] else 0,
                                    q_stride=st["qs"], kv_stride=st["kvs"])
    if c["kind"] == "rope":
        st["shape"] = m.rope_shape(T, Hq, Hkv, D, q_stride=st["qs"], k_stride=st["kvs"])
        st["ko"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    if c["kind"] in ("rope", "append"):
        st["qo"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    elif c["kind"] == "attn":
        st["o"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        st["ws"] = m.paged_alloc_workspace(st["shape"], dev)
    else:
        st["lens_out"] = torch.empty_like(st["starts"])


# --------------------------------------------------------------------- run ---

def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    if c["kind"] == "rope":
        return dict(q=_turned(st, st["q"], st["q_gain"], st["positions"]),
                    k=_turned(st, st["kn"], st["k_gain"], st["positions"]))
    if c["kind"] == "append":
        b, at = _tokens(st)
        pos = st["positions"] if c["tree"] else at
        pages, row = st["tables"][b, at // c["page"]].long(), at % c["page"]
        st["k_pages"][pages, :, row] = _turned(st, st["kn"], st["k_gain"], pos)
        st["v_pages"][pages, :, row] = st["vn"]
        return dict(q=_turned(st, st["q"], st["q_gain"], pos), k_pages=st["k_pages"], v_pages=st["v_pages"])
    if c["kind"] == "attn":
        return dict(o=_attend(st))
    return _keep(st)


def _run_own(st):
    m, c = st["m"], st["case"]
    if c["kind"] == "rope":
        m.rope(st["shape"], st["spec"], st["q"], st["kn"], st["positions"], st["qo"], st["ko"])
        return dict(q=st["qo"], k=st["ko"])
    if c["kind"] == "append":
        m.paged_append(st["shape"], st["spec"], st["q"], st["kn"], st["vn"], st["offsets"], st["starts"], st["cache"],
                       st["qo"], positions=st["positions"] if c["tree"] else None)
        return dict(q=st["qo"], k_pages=st["k_pages"], v_pages=st["v_pages"])
    if c["kind"] == "attn":
        m.paged_attn(st["shape"], st["q"], st["cache"], st["offsets"], st["lens"], st["o"], st["ws"],
                     tree=st["tree"] if c["tree"] else None)
        return dict(o=st["o"])
    m.paged_keep(st["shape"], st["cache"], st["starts"], st["kept"], st["path"], lens_out=st["lens_out"])
    return dict(k_pages=st["k_pages"], v_pages=st["v_pages"], lens=st["lens_out"])


# -------------------------------------------------------------- plain form ---

def _tokens(st):
    """The sequence and position of every packed token."""
    t = torch.arange(st["T"], device=st["dev"])
    b = torch.bucketize(t, st["offsets"][1:], right=True)
    return b, (st["starts"][b] + t - st["offsets"][b]).long()


def _turned(st, x, gain, pos):
    c = st["case"]
    rot, h = c["rot"], c["rot"] // 2
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (c["offset"] + gain.float())
    angle = pos.double().unsqueeze(1) * st["w"]
    cos = (angle.cos() * st["magnitude"]).float().unsqueeze(1)
    sin = (angle.sin() * st["magnitude"]).float().unsqueeze(1)
    if c["layout"] == "half":
        a, b = x[..., :h], x[..., h:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1).to(torch.bfloat16)


def _rows(st, pages):
    """Every sequence's cached rows, fp32 [B, Hkv, P * page, D] (any values past its length)."""
    x = pages[st["tables"].clamp_min(0).long()].float()  # [B, P, Hkv, page, D]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attend(st):
    c = st["case"]
    B, N, Hq, Hkv, D = st["B"], st["nmax"], c["Hq"], c["Hkv"], c["D"]
    r = Hq // Hkv
    K, V = _rows(st, st["k_pages"]), _rows(st, st["v_pages"])
    L = K.shape[2]
    i = torch.arange(N, device=K.device)
    off, n = st["offsets"][:-1].long(), st["offsets"].diff().long()
    row = (off.unsqueeze(1) + i).clamp_max(st["T"] - 1)
    q = st["q"][row].float()  # [B, N, Hq, D], padded
    q = q.view(B, N, Hkv, r, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, r * N, D)
    s = torch.matmul(q, K.transpose(2, 3)).view(B, Hkv, r, N, L) * (1.0 / math.sqrt(D))
    first = st["lens"].long() - n  # the first new token's position
    j = torch.arange(L, device=K.device)
    hidden = j > (first.unsqueeze(1) + i).unsqueeze(2)  # [B, N, L]
    if c["tree"]:
        d = (j - first.unsqueeze(1)).unsqueeze(1).expand(B, N, L)  # the draft at position j
        words = st["tree"][row]  # [B, N, W]
        bit = words.gather(2, (d // 64).clamp(0, st["words"] - 1)) >> (d % 64) & 1
        hidden = hidden | ((d >= 0) & (bit == 0))
    s.masked_fill_(hidden[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, r * N, L), V).view(B, Hkv, r, N, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    t = torch.arange(st["T"], device=K.device)
    b = torch.bucketize(t, st["offsets"][1:], right=True)
    return o[b, t - off[b]].to(torch.bfloat16)


def _keep(st):
    page = st["case"]["page"]
    k = torch.arange(st["path"].shape[1], device=st["dev"])
    b, k = torch.nonzero(k < st["kept"].unsqueeze(1), as_tuple=True)
    src, dst = st["starts"][b] + st["path"][b, k], st["starts"][b] + k
    for pages in (st["k_pages"], st["v_pages"]):
        rows = pages[st["tables"][b, src // page].long(), :, (src % page).long()]
        pages[st["tables"][b, dst // page].long(), :, dst % page] = rows
    return dict(k_pages=st["k_pages"], v_pages=st["v_pages"], lens=st["starts"] + st["kept"])


# -------------------------------------------------------------------- work ---

def work(case):
    Hq, Hkv, D, kind = case["Hq"], case["Hkv"], case["D"], case["kind"]
    if kind == "rope":
        return dict(bytes=4 * case["T"] * (Hq + Hkv) * D, flops=4 * case["T"] * (Hq + Hkv) * D)
    lens, news = _ints(case["lens"]), _ints(case["news"])
    T = sum(news)
    if kind == "append":
        return dict(bytes=4 * T * (Hq + 2 * Hkv) * D, flops=4 * T * (Hq + Hkv) * D)
    if kind == "keep":
        return dict(bytes=8 * sum(_ints(case["kept"])) * Hkv * D, flops=0)
    seen = sum(n for n, m in zip(lens, news) if m)
    # of a tree of m drafts a draft sees about log2(m) + 1 of them
    pairs = sum(m * (n - m) + (m * m.bit_length() if case["tree"] else m * (m + 1) // 2) for n, m in zip(lens, news))
    return dict(bytes=4 * Hkv * seen * D + 4 * T * Hq * D, flops=4 * Hq * D * pairs)


# ------------------------------------------------------------------- exact ---

def _turned64(st, x, gain, pos):
    """The same in complex numbers, fp64: each pair times e^(i angle)."""
    c = st["case"]
    rot = c["rot"]
    x = x.double()
    if c["norm"]:
        size = torch.sqrt((x * x).sum(-1) / x.shape[-1] + EPS)
        x = x / size.unsqueeze(-1) * (gain.double() + c["offset"])
    re, im = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["layout"] == "pairs" else x[..., :rot].chunk(2, -1)
    angle = pos.double()[:, None, None] * st["w"]
    z = torch.complex(re.contiguous(), im.contiguous()) * torch.polar(torch.full_like(angle, st["magnitude"]), angle)
    if c["layout"] == "pairs":
        turned = torch.view_as_real(z).reshape(*z.shape[:-1], rot)
    else:
        turned = torch.cat((z.real, z.imag), -1)
    x = x.clone()
    x[..., :rot] = turned
    return x


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return dict(q=_turned64(st, st["q"], st["q_gain"], st["positions"]),
                    k=_turned64(st, st["kn"], st["k_gain"], st["positions"]))
    lens, news, page = _ints(case["lens"]), _ints(case["news"]), case["page"]
    tables = st["tables"].tolist()
    if kind == "attn":
        return dict(o=_exact_attn(st, tables, lens, news))
    k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
    if kind == "append":
        b, at = _tokens(st)
        pos = st["positions"] if case["tree"] else at
        k, v = _turned64(st, st["kn"], st["k_gain"], pos), st["vn"].double()
        t = 0
        for table, n, m in zip(tables, lens, news):
            p = n - m
            while p < n:  # one page at a time
                end = min(n, (p // page + 1) * page)
                for pages, x in ((k_pages, k), (v_pages, v)):
                    pages[table[p // page], :, p % page:p % page + end - p] = x[t:t + end - p].transpose(0, 1)
                t += end - p
                p = end
        return dict(q=_turned64(st, st["q"], st["q_gain"], pos), k_pages=k_pages, v_pages=v_pages)
    path, after = st["path"].tolist(), []
    for table, n, m, kept, steps in zip(tables, lens, news, _ints(case["kept"]), path):
        s = n - m
        for i, j in enumerate(steps[:kept]):
            if i != j:
                for pages in (k_pages, v_pages):
                    pages[table[(s + i) // page], :, (s + i) % page] = pages[table[(s + j) // page], :, (s + j) % page]
        after.append(s + kept)
    return dict(k_pages=k_pages, v_pages=v_pages, lens=torch.tensor(after, dtype=torch.int32, device=st["dev"]))


def _exact_attn(st, tables, lens, news):
    c = st["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    r = Hq // Hkv
    q, at, rows = st["q"].double(), 0, []
    for table, n, m in zip(tables, lens, news):
        if m == 0:
            continue
        own_pages = torch.tensor(table[:-(-n // page)], device=q.device)
        see = torch.ones(m, n, dtype=torch.bool, device=q.device).tril(n - m)
        if c["tree"]:
            words = st["tree"][at:at + m].cpu().numpy().view(np.uint8)  # little-endian bits
            bits = np.unpackbits(words.reshape(m, -1), axis=1, bitorder="little")[:, :m].astype(bool)
            see[:, n - m:] &= torch.from_numpy(bits).to(q.device)
        out = torch.zeros(m, Hq, D, dtype=torch.float64, device=q.device)
        for g in range(Hkv):
            K = st["k_pages"][own_pages, g].reshape(-1, D)[:n].double()
            V = st["v_pages"][own_pages, g].reshape(-1, D)[:n].double()
            for i in range(0, m, 512):
                x = q[at + i:at + min(m, i + 512), g * r:(g + 1) * r]
                w = torch.einsum("thd,jd->thj", x, K) / math.sqrt(D)
                w = torch.softmax(w.masked_fill(~see[i:i + x.shape[0]].unsqueeze(1), -math.inf), -1)
                out[i:i + x.shape[0], g * r:(g + 1) * r] = torch.einsum("thj,jd->thd", w, V)
        rows.append(out)
        at += m
    return torch.cat(rows)
