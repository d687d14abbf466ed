"""The operators of a tree-drafted decoding step over the NVFP4 cache, as they
are measured: norms + rotation + quantizing append, tree attention,
verification of the drafts, and keeping the accepted path's cache slots.

`run` computes them in elementary torch operations where `own` is false, and
calls the package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user, a short conversation, four drafted tokens in a chain: latency
        dict(name="tree_short", op="tree", B=1, Hq=32, Hkv=8, D=128, N=4, lo=300, hi=300, paged=False, out="bf16",
             mask="chain", nodes="full"),
        # the GQA decode workload's sizes with a 16-node tree, paged
        dict(name="tree_gqa_paged", op="tree", B=8, Hq=32, Hkv=8, D=128, N=16, lo=4096, hi=4096, paged=True,
             out="bf16", mask="tree", nodes="full"),
        # the large ragged batch, 8-node trees of which some hold fewer nodes
        dict(name="tree_ragged", op="tree", B=128, Hq=32, Hkv=8, D=128, N=8, lo=1024, hi=8192, paged=False,
             out="bf16", mask="tree", nodes="ragged"),
        # one 64K context, a wide tree: 256 rows a KV head
        dict(name="tree_long64k", op="tree", B=1, Hq=64, Hkv=8, D=128, N=32, lo=65536, hi=65536, paged=False,
             out="bf16", mask="tree", nodes="full"),
        # 128K context, GQA group 12, fp32 outputs
        dict(name="tree_128k_f32", op="tree", B=1, Hq=96, Hkv=8, D=128, N=16, lo=131072, hi=131072, paged=False,
             out="f32", mask="tree", nodes="full"),
        # one new token of each of eight sequences in front of decode attention: latency
        dict(name="append_decode", op="append", B=8, Hq=32, Hkv=8, D=128, n=1, R=128, dtype="bf16", paged=False,
             interleaved=False, norm=True, nodes="full", depth=False, packed=True),
        # the nodes of a ragged batch of trees into a paged cache, positions by depth
        dict(name="append_tree_paged", op="append", B=128, Hq=32, Hkv=8, D=128, n=8, R=64, dtype="bf16", paged=True,
             interleaved=False, norm=True, nodes="ragged", depth=True, packed=True),
        # a 2048-token prompt chunk of the 96-head workload, interleaved pairs
        dict(name="append_chunk", op="append", B=1, Hq=96, Hkv=8, D=128, n=2048, R=128, dtype="bf16", paged=False,
             interleaved=True, norm=True, nodes="full", depth=False, packed=False),
        # a chain of five drafts for one user
        dict(name="verify_chain", op="verify", B=1, N=6, V=32000, dtype="f32", tree="chain", draft=True,
             nodes="full"),
        # trees of sixteen nodes for a batch, with the draft's distributions
        dict(name="verify_tree", op="verify", B=64, N=16, V=131072, dtype="f32", tree="tree", draft=True,
             nodes="ragged"),
        # sixteen layers' K and V after a step of eight sequences
        dict(name="commit_layers", op="commit", layers=16, B=8, Hkv=8, D=128, S=512, N=16, paged=False),
        # a large paged batch, four layers
        dict(name="commit_paged", op="commit", layers=4, B=128, Hkv=8, D=128, S=256, N=32, paged=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "append", "verify", "commit"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    if op == "tree":
        B = _logint(rng, 1, 64)
        N = _logint(rng, 1, 64)
        hi = _logint(rng, 1, max(1, min(65536, (1 << 22) // (B * Hkv), (1 << 29) // (B * Hkv * g * N))))
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, D=D, N=N, lo=rng.randint(0, hi), hi=hi, paged=rng.random() < 0.4,
                    out=rng.choice(["bf16", "f32"]), mask=rng.choice(["tree", "tree", "chain"]),
                    nodes=rng.choice(["full", "ragged"]))
    if op == "append":
        B = _logint(rng, 1, 128)
        n = _logint(rng, 1, max(1, min(2048, 8192 // (B * Hkv))))
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, D=D, n=n, R=rng.choice([D, D, D // 2, 16, 48]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), paged=rng.random() < 0.4,
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8, nodes=rng.choice(["full", "ragged"]),
                    depth=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "verify":
        B = _logint(rng, 1, 64)
        N = _logint(rng, 1, 24)
        V = _logint(rng, 1000, min(200000, (1 << 27) // (B * N)))
        return dict(op=op, B=B, N=N, V=V, dtype=rng.choice(["f32", "f32", "bf16"]),
                    tree=rng.choice(["tree", "chain"]), draft=rng.random() < 0.7, nodes=rng.choice(["full", "ragged"]))
    N = _logint(rng, 1, 64)
    return dict(op=op, layers=rng.randint(1, 16), B=_logint(rng, 1, 32), Hkv=Hkv, D=D,
                S=128 * rng.randint(1, 3), N=N, paged=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# what is the same for every seed of a case: lengths, counts, trees
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers of [lo, hi], both ends among them, in a mixed order."""
    if n == 1:
        return [hi]
    return [lo + ((hi - lo) * ((i * 37) % n)) // (n - 1) if n % 37 else lo + ((hi - lo) * i) // (n - 1)
            for i in range(n)]


def _counts(case, n):
    """Nodes (new tokens) of each sequence."""
    if case["nodes"] == "full":
        return [n] * case["B"]
    return [max(1, n - (i * 5) % n) if i % 7 else n for i in range(case["B"])]


def _starts(case):
    return _spread(case["lo"], case["hi"], case["B"])


def _parents(kind, n):
    """Parent of each node, -1 for the root; a node comes after its parent."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    return [-1] + [(i - 1) // 2 if i % 3 else max(0, i - 2) for i in range(1, n)]


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _ancestors(parents):
    """Bool [n][n]: node i sees node j (itself and its ancestors)."""
    n = len(parents)
    m = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def _mask_words(m):
    n = m.shape[0]
    w = np.zeros((n, (n + 31) // 32), np.uint32)
    for j in range(n):
        w[:, j // 32] |= m[:, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(w.view(np.int32)).to(DEV)


# ---------------------------------------------------------------------------
# NVFP4 in elementary operations
# ---------------------------------------------------------------------------
_MIDS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def _quantize(x, s):
    """Codes [..., D/2] and scale bytes [..., D/16] of x [..., D] (fp32), tensor scale s (fp32 tensor)."""
    shape = x.shape
    x = x.reshape(*shape[:-1], shape[-1] // 16, 16)
    r = x.abs().amax(-1) / (s * 6.0)
    sb = r.clamp(max=448.0).to(torch.float8_e4m3fn)
    den = (sb.float() * s).unsqueeze(-1)
    y = torch.where(den == 0, torch.zeros_like(x), x / den)
    # ties go to the even code: above 0.25, from 0.75, above 1.25, ...
    edges = torch.tensor(_MIDS, device=x.device)
    edges[1::2] = torch.nextafter(edges[1::2], torch.zeros_like(edges[1::2]))
    code = torch.bucketize(y.abs(), edges, out_int32=True) + 8 * torch.signbit(x)
    code = code.to(torch.uint8).reshape(*shape[:-1], shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), sb.view(torch.uint8).reshape(*shape[:-1], shape[-1] // 16)


def _fp8_values(codes, scales, s):
    """The FP8 values (float8) that codes [..., D/2] and scales [..., D/16] stand for."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1, 16)
    v = grid[(c & 7).int()] * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1) * s
    v = torch.where(c >= 8, -v, v).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _gather_pages(pool, table):
    """[pages][H][T][X] and a table [B][M] -> [B][H][M * T][X]."""
    B, M = table.shape
    _, H, T, X = pool.shape
    return pool[table.long()].permute(0, 2, 1, 3, 4).reshape(B, H, M * T, X)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(gen, B, Hkv, S, D):
    """Codes, scale bytes and tensor scale of a cache of N(0,1) values times log-normal channel scales."""
    ch = torch.exp(torch.randn(Hkv, 1, D, generator=gen, device=DEV) * 0.5)
    s = (ch.amax() * 6.0 / 2688.0).reshape(1)
    codes = torch.empty(B, Hkv, S, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(B, Hkv, S, D // 16, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (Hkv * S * D))
    for b in range(0, B, step):
        x = torch.randn(min(step, B - b), Hkv, S, D, generator=gen, device=DEV) * ch
        codes[b:b + step], scales[b:b + step] = _quantize(x, s)
    return codes, scales, s


def _pages(gen, B, capacity):
    """A block table [B][M] of 128-token pages in a mixed order."""
    M = -(-capacity // 128)
    return torch.randperm(B * M, generator=gen, device=DEV).to(torch.int32).reshape(B, M).contiguous(), M


def _prepare_tree(case, gen):
    B, Hkv, D, N = case["B"], case["Hkv"], case["D"], case["N"]
    starts, counts = _starts(case), _counts(case, N)
    cap = max(starts) + N
    s = dict(case=case, start=_int32(starts), nodes=None if case["nodes"] == "full" else _int32(counts))
    if case["paged"]:
        s["table"], M = _pages(gen, B, cap)
        kc, ks, s["sk"] = _cache(gen, B * M, Hkv, 128, D)
        vc, vs, s["sv"] = _cache(gen, B * M, Hkv, 128, D)
    else:
        S = -(-cap // 16) * 16
        kc, ks, s["sk"] = _cache(gen, B, Hkv, S, D)
        vc, vs, s["sv"] = _cache(gen, B, Hkv, S, D)
    s.update(kc=kc, ks=ks, vc=vc, vs=vs)
    s["q"] = torch.randn(B, N, case["Hq"], D, generator=gen, device=DEV).to(torch.bfloat16)
    s["mask"] = None if case["mask"] == "chain" else _mask_words(_ancestors(_parents("tree", N)))
    s["out"] = torch.zeros(B, N, case["Hq"], D, device=DEV,
                           dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if own:
        import bit_decode_attention_b200 as nv
        s["ws"] = torch.zeros(nv.nvfp4_tree_attention_workspace(B, N, case["Hq"], Hkv, D), dtype=torch.uint8,
                              device=DEV)
    return s


def _prepare_append(case, gen):
    B, Hq, Hkv, D, n, R = (case[k] for k in ("B", "Hq", "Hkv", "D", "n", "R"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    ch = torch.exp(torch.randn(Hq + 2 * Hkv, D, generator=gen, device=DEV) * 0.5)
    x = (torch.randn(B, n, Hq + 2 * Hkv, D, generator=gen, device=DEV) * ch).to(dt)
    parts = [x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]]
    if not case["packed"]:
        parts = [p.contiguous() for p in parts]
    starts = [(i * 7) % 33 for i in range(B)]
    counts = _counts(case, n)
    depth = _depths(_parents("tree", n))
    s = dict(case=case, xq=parts[0], xk=parts[1], xv=parts[2], start=_int32(starts),
             counts=None if case["nodes"] == "full" else _int32(counts),
             positions=_int32([[5000 + st + d for d in depth] for st in starts]) if case["depth"] else None)
    cap = max(starts) + n
    # cos and sin of a long context's positions, angles in 64 bits
    P = 16384
    inv = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
    ang = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * inv
    s["table_cs"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    wq, wk = (1.0 + 0.2 * torch.randn(2, D, generator=gen, device=DEV)).to(dt)
    s["wq"], s["wk"] = (wq.contiguous(), wk.contiguous()) if case["norm"] else (None, None)
    s["sk"] = torch.tensor([11.3719 / 2688.0], device=DEV)
    s["sv"] = torch.tensor([19.5377 / 2688.0], device=DEV)
    if case["paged"]:
        s["pages"], M = _pages(gen, B, cap)
        dims = (B * M, Hkv, 128)
        # every slot of every page is read back
        s["lens"] = torch.full((B * M,), 128, dtype=torch.int32, device=DEV)
    else:
        S = -(-cap // 16) * 16
        dims = (B, Hkv, S)
        s["lens"] = torch.full((B,), S, dtype=torch.int32, device=DEV)
    for p in ("k", "v"):
        s[p + "c"] = torch.zeros(*dims, D // 2, dtype=torch.uint8, device=DEV)
        s[p + "s"] = torch.zeros(*dims, D // 16, dtype=torch.uint8, device=DEV)
        s[p + "8"] = torch.zeros(*dims, D, dtype=torch.uint8, device=DEV)
    s["q_out"] = torch.zeros(B, n, Hq, D, dtype=dt, device=DEV)
    s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    return s


def _prepare_verify(case, gen):
    B, N, V = case["B"], case["N"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # the draft's logits are the target's with noise, both peaked as a language model's
    base = torch.randn(B, N, V, generator=gen, device=DEV) * 2.5
    target = torch.softmax(base, -1).to(dt)
    noisy = base.add_(torch.randn(B, N, V, generator=gen, device=DEV), alpha=0.7)
    draft = torch.softmax(noisy, -1).to(dt)
    del base, noisy
    parents = _parents(case["tree"], N)
    up = torch.tensor([max(p, 0) for p in parents], device=DEV)
    # a node's token is drawn from the draft's distribution at its parent
    u = torch.rand(B, N, generator=gen, device=DEV, dtype=torch.float64)
    tokens = torch.empty(B, N, dtype=torch.int32, device=DEV)
    for i in range(N):
        c = draft[:, int(up[i])].double().cumsum(-1)
        tokens[:, i] = (c <= u[:, i:i + 1] * c[:, -1:]).sum(-1).clamp(max=V - 1)
    s = dict(case=case, p=target, d=draft if case["draft"] else None, tokens=tokens, parents=_int32(parents),
             plist=parents, ua=torch.rand(B, N, generator=gen, device=DEV),
             us=torch.rand(B, generator=gen, device=DEV),
             counts=None if case["nodes"] == "full" else _int32(_counts(case, N)))
    s["path"] = torch.zeros(B, N, dtype=torch.int32, device=DEV)
    s["n_acc"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    s["next"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    return s


def _prepare_commit(case, gen):
    L, B, Hkv, D, S, N = (case[k] for k in ("layers", "B", "Hkv", "D", "S", "N"))
    s = dict(case=case)
    dims = (2 * L, B, Hkv, S)
    cap = S
    if case["paged"]:
        s["pages"], M = _pages(gen, B, S)
        dims = (2 * L, B * M, Hkv, 128)
        cap = 128 * M
    s["codes"] = torch.randint(0, 256, (*dims, D // 2), generator=gen, device=DEV, dtype=torch.uint8)
    s["scales"] = torch.randint(0, 127, (*dims, D // 16), generator=gen, device=DEV, dtype=torch.uint8)
    s["start"] = torch.randint(0, cap - N + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
    # paths of one to about eight nodes: the root, then nodes in growing order
    keep = torch.rand(B, N, generator=gen, device=DEV) < min(0.5, 6.0 / N)
    keep[:, 0] = True
    order = torch.where(keep, 0, 1) * N + torch.arange(N, device=DEV)
    path = order.sort(-1).values
    s["path"] = torch.where(path < N, path, -1).to(torch.int32)
    s["n_acc"] = keep.sum(-1).to(torch.int32)
    s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    s = {"tree": _prepare_tree, "append": _prepare_append, "verify": _prepare_verify,
         "commit": _prepare_commit}[op](case, gen)
    if own:
        import bit_decode_attention_b200 as nv
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op in ("tree", "append"):
            table = s.get("table", s.get("pages"))
            s["k"], s["v"] = (nv.PagedKVPlane(s[p + "c"], s[p + "s"], table) if table is not None
                              else nv.KVPlane(s[p + "c"], s[p + "s"]) for p in ("k", "v"))
        if op == "append":
            # the pool's pages read back as sequences of one page each
            s["k_read"], s["v_read"] = (nv.KVPlane(s[p + "c"], s[p + "s"]) for p in ("k", "v"))
        if op == "commit":
            s["planes"] = nv.KVPlaneList(nv.PagedKVPlane(c, t, s["pages"]) if case["paged"] else nv.KVPlane(c, t)
                                         for c, t in zip(s["codes"], s["scales"]))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _visible(s, S):
    """Bool [B][N][S]: what each node sees."""
    N = s["case"]["N"]
    t = torch.arange(S, device=DEV)
    i = torch.arange(N, device=DEV)
    rel = t[None, :] - s["start"][:, None]
    inside = (rel >= 0) & (rel < N)
    j = rel.clamp(0, N - 1)
    if s["mask"] is None:
        seen = j[:, None, :] <= i[None, :, None]
    else:
        bits = ((s["mask"][:, :, None] >> torch.arange(32, device=DEV)) & 1).reshape(N, -1).bool()
        seen = bits[i[None, :, None], j[:, None, :]]
    return (rel < 0)[:, None, :] | (inside[:, None, :] & seen)


def _tree(s):
    c = s["case"]
    if own:
        import bit_decode_attention_b200 as nv
        call = nv.nvfp4_tree_attention_paged if c["paged"] else nv.nvfp4_tree_attention
        return call(s["q"], s["k"], s["v"], s["sk"], s["sv"], s["start"], tree_mask=s["mask"], n_nodes=s["nodes"],
                    out=s["out"], workspace=s["ws"], status=s["status"])
    B, N, Hq, D = s["q"].shape
    Hkv, g = c["Hkv"], Hq // c["Hkv"]
    kc, ks, vc, vs = ((_gather_pages(s[x], s["table"]) if c["paged"] else s[x]) for x in ("kc", "ks", "vc", "vs"))
    k = _fp8_values(kc, ks, s["sk"]).float()
    q = s["q"].float().reshape(B, N, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * g, D)
    scores = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    del k
    hidden = ~_visible(s, scores.shape[-1])[:, None, :, None, :]
    scores = scores.reshape(B, Hkv, N, g, -1).masked_fill_(hidden, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    del scores
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, N * g, -1), _fp8_values(vc, vs, s["sv"]).float()).reshape(B, Hkv, N, g, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["out"].dtype)
    if s["nodes"] is None:
        return o
    live = torch.arange(N, device=DEV)[None, :] < s["nodes"][:, None]
    return torch.where(live[:, :, None, None], o, s["out"])


def _norm_rope(x, w, norm, cs, pos, interleaved):
    x = x.float()
    if norm:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    R = cs.shape[1]
    cos, sin = cs[pos.long()][:, :, None, :].split(R // 2, -1)
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, x[..., R:]], -1)


def _append(s):
    c = s["case"]
    eps = 1e-6 if c["norm"] else -1.0
    if own:
        import bit_decode_attention_b200 as nv
        call = nv.nvfp4_qk_norm_rope_append_paged if c["paged"] else nv.nvfp4_qk_norm_rope_append
        q = call(s["xq"], s["xk"], s["xv"], s["start"], s["sk"], s["sv"], s["k"], s["v"], w_q=s["wq"], w_k=s["wk"],
                 eps=eps, rope_table=s["table_cs"], interleaved=c["interleaved"], positions=s["positions"],
                 n_valid=s["counts"], q_out=s["q_out"], new_lens=s["new_lens"], status=s["status"])
        nv.nvfp4_kv_dequant_fp8(s["k_read"], s["sk"], s["lens"], out=s["k8"])
        nv.nvfp4_kv_dequant_fp8(s["v_read"], s["sv"], s["lens"], out=s["v8"])
        return [q, s["new_lens"], s["k8"].view(torch.float8_e4m3fn), s["v8"].view(torch.float8_e4m3fn)]
    B, n, Hq, D = s["xq"].shape
    i = torch.arange(n, device=DEV)
    slots = s["start"][:, None] + i
    pos = s["positions"] if s["positions"] is not None else slots
    q = _norm_rope(s["xq"], s["wq"], c["norm"], s["table_cs"], pos, c["interleaved"]).to(s["xq"].dtype)
    k = _norm_rope(s["xk"], s["wk"], c["norm"], s["table_cs"], pos, c["interleaved"])
    counts = s["counts"] if s["counts"] is not None else torch.full((B,), n, dtype=torch.int32, device=DEV)
    b, j = (i[None, :] < counts[:, None]).nonzero(as_tuple=True)
    t = slots[b, j].long()
    seq = b if not c["paged"] else s["pages"][b, t // 128].long()
    t = t if not c["paged"] else t % 128
    for p, x, st in (("k", k, s["sk"]), ("v", s["xv"].float(), s["sv"])):
        codes, scales = _quantize(x[b, j], st)
        s[p + "c"][seq, :, t] = codes
        s[p + "s"][seq, :, t] = scales
    live = (i[None, :] < counts[:, None])[:, :, None, None]
    return [torch.where(live, q, s["q_out"]), s["start"] + counts, _fp8_values(s["kc"], s["ks"], s["sk"]),
            _fp8_values(s["vc"], s["vs"], s["sv"])]


def _verify(s):
    c = s["case"]
    if own:
        import bit_decode_attention_b200 as nv
        return nv.nvfp4_verify_drafts(s["p"], s["d"], s["tokens"], s["parents"], s["ua"], s["us"], n_nodes=s["counts"],
                                      path=s["path"], n_accepted=s["n_acc"], next_token=s["next"], status=s["status"])
    B, N, V = s["p"].shape
    rows = torch.arange(B, device=DEV)
    counts = s["counts"] if s["counts"] is not None else torch.full((B,), N, device=DEV)
    at = torch.zeros(B, dtype=torch.long, device=DEV)
    path = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    n_acc = torch.ones(B, dtype=torch.int32, device=DEV)
    w = s["p"][:, 0].double()
    Z = torch.ones(B, dtype=torch.float64, device=DEV)
    # a node comes after its parent and siblings are tried in order: one walk over the nodes
    for i in range(1, N):
        tested = (at == s["plist"][i]) & (i < counts)
        x = s["tokens"][:, i].long()
        d = (s["d"][rows, at].double() if s["d"] is not None
             else torch.nn.functional.one_hot(x, V).double())
        taken = tested & (s["ua"][:, i].double() * d[rows, x] * Z < w[rows, x])
        rest = (w - Z[:, None] * d).clamp(min=0)
        total = rest.sum(-1)
        kept = (tested & ~taken & (total > 0))[:, None]
        w = torch.where(taken[:, None], s["p"][:, i].double(), torch.where(kept, rest, w))
        Z = torch.where(taken, 1.0, torch.where(kept[:, 0], total, Z))
        path[rows, n_acc] = torch.where(taken, i, -1).to(torch.int32)
        n_acc += taken.int()
        at = torch.where(taken, i, at)
    cum = w.cumsum(-1)
    token = (cum <= s["us"].double()[:, None] * cum[:, -1:]).sum(-1).clamp(max=V - 1).to(torch.int32)
    return [path, n_acc, token]


def _commit(s):
    c = s["case"]
    if own:
        import bit_decode_attention_b200 as nv
        call = nv.nvfp4_kv_commit_path_paged if c["paged"] else nv.nvfp4_kv_commit_path
        call(s["planes"], s["start"], s["path"], s["n_acc"], new_lens=s["new_lens"], status=s["status"])
        return [s["codes"], s["scales"], s["new_lens"]]
    N = c["N"]
    b, j = (torch.arange(N, device=DEV)[None, :] < s["n_acc"][:, None]).nonzero(as_tuple=True)
    src = (s["start"][b] + s["path"][b, j]).long()
    dst = (s["start"][b] + j).long()
    sb, db = (b, b) if not c["paged"] else (s["pages"][b, src // 128].long(), s["pages"][b, dst // 128].long())
    if c["paged"]:
        src, dst = src % 128, dst % 128
    s["codes"][:, db, :, dst] = s["codes"][:, sb, :, src]
    s["scales"][:, db, :, dst] = s["scales"][:, sb, :, src]
    return [s["codes"], s["scales"], s["start"] + s["n_acc"]]


def run(state):
    return {"tree": _tree, "append": _append, "verify": _verify, "commit": _commit}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "tree":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        starts, counts = _starts(case), _counts(case, case["N"])
        esz = 2 if case["out"] == "bf16" else 4
        tokens = sum(a + n for a, n in zip(starts, counts))
        nodes = sum(counts)
        anc = _ancestors(_parents("tree" if case["mask"] == "tree" else "chain", case["N"])).sum(1)
        pairs = sum(n * a + int(anc[:n].sum()) for a, n in zip(starts, counts))
        return dict(bytes=2 * tokens * Hkv * (D // 2 + D // 16) + nodes * Hq * D * (2 + esz), flops=4 * D * Hq * pairs)
    if op == "append":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        esz = 2 if case["dtype"] == "bf16" else 4
        n = sum(_counts(case, case["n"]))
        slots = -(-(max((i * 7) % 33 for i in range(case["B"])) + case["n"]) // (128 if case["paged"] else 16))
        slots *= (128 if case["paged"] else 16) * case["B"]
        # the step itself, and the read-back of both planes as FP8
        own_bytes = n * ((2 * Hq + 2 * Hkv) * D * esz + 2 * Hkv * (D // 2 + D // 16) + 4 * case["R"])
        return dict(bytes=own_bytes + 2 * slots * Hkv * (D // 2 + D // 16 + D), flops=10 * n * (Hq + 2 * Hkv) * D)
    if op == "verify":
        esz = 2 if case["dtype"] == "bf16" else 4
        rows = 2 if case["draft"] else 1
        return dict(bytes=case["B"] * (case["V"] * esz * rows + case["N"] * 20), flops=3 * case["B"] * case["V"] * rows)
    moved = case["layers"] * 2 * case["B"] * max(1, min(6, case["N"] // 2)) * case["Hkv"] * (case["D"] // 2 +
                                                                                            case["D"] // 16)
    return dict(bytes=2 * moved, flops=0)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_grid():
    """The 127 non-negative E4M3 values in byte order."""
    return np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])


def _near(x, grid):
    """Index of the grid value nearest to x >= 0 (64 bits), ties to the even index, saturating."""
    g = torch.as_tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(g, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = g[hi] - x, x - g[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def _fp8_table(s):
    """FP8 value of (scale byte, magnitude), from the two fp32 roundings and the nearest E4M3 value."""
    grid = _e4m3_grid()
    mags = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    prod = (grid[:, None] * mags).astype(np.float32) * np.float32(s)
    at = _near(torch.from_numpy(prod.astype(np.float64)), grid)
    return torch.from_numpy(grid)[at].to(DEV)


def _exact_fp8(codes, scales, table):
    nib = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    byte = scales.long().repeat_interleave(16, -1)
    return table[byte, nib % 8] * (1 - 2 * (nib // 8))


def _exact_tree(case, s):
    B, N, Hq, D = s["q"].shape
    Hkv, g = case["Hkv"], Hq // case["Hkv"]
    starts, counts = _starts(case), _counts(case, N)
    tk, tv = _fp8_table(s["sk"].item()), _fp8_table(s["sv"].item())
    seen = _ancestors(_parents("tree" if case["mask"] == "tree" else "chain", N))
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        L = starts[b] + counts[b]
        for h in range(Hkv):
            if case["paged"]:
                pages = s["table"][b].long()
                rows = [s[x][pages, h].reshape(-1, s[x].shape[-1])[:L] for x in ("kc", "ks", "vc", "vs")]
            else:
                rows = [s[x][b, h, :L] for x in ("kc", "ks", "vc", "vs")]
            k = _exact_fp8(rows[0], rows[1], tk).double()
            v = _exact_fp8(rows[2], rows[3], tv).double()
            q = s["q"][b, :counts[b], h * g:(h + 1) * g].double().reshape(-1, D)
            z = (q @ k.T) / math.sqrt(D)
            tail = torch.from_numpy(~seen[:counts[b], :counts[b]]).to(DEV).repeat_interleave(g, 0)
            z[:, starts[b]:].masked_fill_(tail, -math.inf)
            out[b, :counts[b], h * g:(h + 1) * g] = (torch.softmax(z, -1) @ v).reshape(counts[b], g, D)
    return out


def _exact_append(case, s):
    B, n, Hq, D = s["xq"].shape
    R, counts = case["R"], _counts(case, n)
    grid4, grid8 = [0, 0.5, 1, 1.5, 2, 3, 4, 6], _e4m3_grid()
    first, second = ((torch.arange(0, R, 2), torch.arange(1, R, 2)) if case["interleaved"]
                     else (torch.arange(0, R // 2), torch.arange(R // 2, R)))
    start = s["start"].long()
    where = (s["positions"] if s["positions"] is not None else s["start"][:, None] + torch.arange(n, device=DEV)).long()
    cs = s["table_cs"][where].double()[:, :, None]

    def turned(x, w):
        x = x.double()
        if case["norm"]:
            x = x / ((x ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(cs[..., :R // 2], cs[..., R // 2:])
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q = turned(s["xq"], s["wq"])
    planes = []
    for x, scale, like in ((turned(s["xk"], s["wk"]), s["sk"], s["kc"]), (s["xv"].double(), s["sv"], s["vc"])):
        st, table = scale.double(), _fp8_table(scale.item())
        blocks = x.reshape(B, n, -1, D // 16, 16)
        byte = _near(blocks.abs().amax(-1) / (6 * st), grid8)[..., None]
        den = torch.as_tensor(grid8, device=DEV)[byte] * st
        mag = torch.where(den > 0, _near(blocks.abs() / den.clamp(min=1e-300), grid4), 0)
        val = table[byte, mag] * torch.sign(blocks)
        val = val.reshape(B, n, -1, D)
        plane = torch.zeros(*like.shape[:-1], D, dtype=torch.float64, device=DEV)
        for b in range(B):
            slots = start[b] + torch.arange(counts[b], device=DEV)
            if case["paged"]:
                plane[s["pages"][b, slots // 128].long(), :, slots % 128] = val[b, :counts[b]]
            else:
                plane[b, :, slots] = val[b, :counts[b]].transpose(0, 1)
        planes.append(plane)
    for b in range(B):
        q[b, counts[b]:] = 0
    return [q, None] + planes


def _exact_verify(case, s):
    B, N = case["B"], case["N"]
    counts = _counts(case, N)
    tokens, ua, us = s["tokens"].cpu().numpy(), s["ua"].cpu().numpy().astype(np.float64), s["us"].cpu().numpy()
    paths, lengths, nexts = np.full((B, N), -1, np.int32), [], []
    for b in range(B):
        path = [0]
        while True:
            a = path[-1]
            w, Z = s["p"][b, a].double().cpu().numpy(), 1.0
            d = s["d"][b, a].double().cpu().numpy() if s["d"] is not None else None
            moved = False
            for c in [c for c in range(a + 1, counts[b]) if s["plist"][c] == a]:
                x = tokens[b, c]
                if ua[b, c] * (d[x] if d is not None else 1.0) * Z < w[x]:
                    path.append(c)
                    moved = True
                    break
                rest = w - Z * d if d is not None else w.copy()
                if d is None:
                    rest[x] -= Z
                rest = np.maximum(rest, 0)
                if math.fsum(rest) > 0:
                    w, Z = rest, math.fsum(rest)
            if not moved:
                break
        paths[b, :len(path)] = path
        lengths.append(len(path))
        c = np.cumsum(w)
        nexts.append(int(np.searchsorted(c, float(us[b]) * c[-1], side="right")))
    return [torch.from_numpy(paths), torch.tensor(lengths, dtype=torch.int32), torch.tensor(nexts, dtype=torch.int32)]


def exact(case, seed):
    if case["op"] == "commit":
        return None  # bytes are moved, nothing is computed
    s = prepare(case, seed)
    return {"tree": _exact_tree, "append": _exact_append, "verify": _exact_verify}[case["op"]](case, s)
