"""The tree-step operators on the GPU at the ends of their documented ranges: nodes and
group sizes up to the limits, values that are no numbers, rows that nobody computes."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import synthetic
import tree_reference as ref
from test_gpu_tree_step import (block_table, check_verify, dev, i32, make_rope, make_verify, run_append, run_tree,
                                status, to_pages)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_decode_attention_b200 as nv
    return nv


def check_cleaned_verify(nv, p, d, tok, par, ua, us):
    """The walk on raw rows against the definition's on rows whose NaN and negatives are 0."""
    st = status()
    path, n_acc, nxt = (t.tolist() for t in nv.nvfp4_verify_drafts(dev(p), dev(d), dev(tok), dev(par), dev(ua), dev(us),
                                                                   status=st))
    clean = lambda t: torch.where(t > 0, t, torch.zeros_like(t)).double().numpy()
    for b in range(p.shape[0]):
        want, token = ref.verify(clean(p[b]), clean(d[b]), tok[b].tolist(), par.tolist(), ua[b].double().numpy(),
                                 float(us[b]), p.shape[1])
        assert path[b] == want + [-1] * (p.shape[1] - len(want)) and n_acc[b] == len(want) and nxt[b] == token
    return st.item(), path


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_draft_entries_that_are_no_probabilities_count_as_nothing(nv, dtype):
    nan, V = float("nan"), 1024
    p, d = torch.zeros(6, 3, V), torch.zeros(6, 3, V)
    p[:, :, 5], p[:, :, 8] = 0.5, 0.5
    d[:, 0, 9] = 1.0
    par = torch.tensor([-1, 0, 0], dtype=torch.int32)
    tok = torch.tensor([[0, 5, 5]] * 6, dtype=torch.int32)
    ua, us = torch.full((6, 3), 0.5), torch.tensor([0.25, 0.75, 0.25, 0.25, 0.75, 0.25])
    d[0, 0, 5] = nan                                       # 0 of the draft's, 0.5 of the target's: accepted
    d[1, 0, 5] = -2.0                                      # likewise
    tok[2, 1], d[2, 0, 7] = 7, -1.0                        # nothing of the target's: not accepted
    tok[2, 2] = 6
    tok[3, 1], d[3, 0, 5] = 9, nan                         # 9 is rejected; 5 keeps its weight beside a NaN
    tok[3, 2] = 6
    tok[4, 1], d[4, 0, 8] = 9, -3.0                        # 8 keeps its weight, no more, beside a negative
    tok[4, 2] = 6
    tok[5, 1], d[5, 0, 7] = 9, -3.0                        # a token without weight gains none
    tok[5, 2] = 6
    st, path = check_cleaned_verify(nv, p.to(dtype), d.to(dtype), tok, par, ua, us)
    assert st == 0 and [q[1] for q in path] == [1, 1, -1, -1, -1, -1]


@pytest.mark.parametrize("N,V,kind", [(9, 4099, "star"), (12, 4096, "tree"), (5, 33000, "star")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_rows_strewn_with_entries_that_are_no_probabilities(nv, N, V, kind, dtype):
    p, d, tok, par, ua, us = make_verify(8, N, V, kind, N + V, dtype)
    g = torch.Generator().manual_seed(V)
    for t in (p, d):
        r = torch.rand(t.shape, generator=g)
        t[r < 0.1] = float("nan")
        t[(r > 0.1) & (r < 0.2)] *= -1.0
    r = torch.rand(8, N, generator=g)
    for b in range(8):                                     # the drafted tokens' own entries too
        for i in range(1, N):
            if r[b, i] < 0.5:
                d[b, par[i], tok[b, i]] = float("nan") if r[b, i] < 0.25 else -0.5
    st, _ = check_cleaned_verify(nv, p, d, tok, par, ua, us)
    assert st == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N,g,D,starts,paged", [
    (4, 4, 128, [60], False), (8, 4, 128, [5000, 1], False), (16, 4, 64, [3000, 130], True), (24, 5, 128, [4000, 9], False),
    (33, 8, 128, [2500, 0], False), (33, 8, 64, [0, 2500], True)])
def test_tree_attention_of_a_query_that_is_no_number(nv, N, g, D, starts, paged, bf16):
    """A query with a NaN or an infinity gives NaN where it sees a token, and nothing to
    the other rows; a node that sees nothing gives zeros whatever its query holds."""
    B, Hkv = len(starts), 2
    S = -(-(max(starts) + N) // 128) * 128
    c, s = synthetic.random_planes(N, B, Hkv, S, D, max_scale_byte=0x50)
    t4 = [c, s, c.flip(2).contiguous(), s.flip(2).contiguous()]
    if paged:
        tbl = block_table(B, S // 128, 3)
        t4 = to_pages(t4, tbl, 128)
        tbl = tbl.cuda()
    t4 = [t.cuda() for t in t4]
    mk = (lambda a, b: nv.PagedKVPlane(a, b, tbl)) if paged else nv.KVPlane
    k, v = mk(t4[0], t4[1]), mk(t4[2], t4[3])
    call = nv.nvfp4_tree_attention_paged if paged else nv.nvfp4_tree_attention
    seen = np.stack([ref.ancestors(ref.parents_of("tree", N))] * B)
    seen[:, N - 1] = False
    q = torch.randn(B, N, g * Hkv, D, generator=torch.Generator().manual_seed(N)).bfloat16().cuda()
    sc, mask, st = torch.tensor([0.01], device="cuda"), dev(ref.mask_words(seen)), status()

    def run(q):
        ws = torch.full((nv.nvfp4_tree_attention_workspace(B, N, g * Hkv, Hkv, D),), 0xFF, dtype=torch.uint8, device="cuda")
        out = call(q, k, v, sc, sc, i32(starts), tree_mask=mask, out_dtype=torch.bfloat16 if bf16 else torch.float32,
                   workspace=ws, status=st)
        assert st.item() == 0
        return out
    want, bad = run(q), torch.zeros(B, N, g * Hkv, dtype=torch.bool)
    assert want.isfinite().all()
    nan, inf = float("nan"), float("inf")
    for i, (value, at) in enumerate([(nan, 0), (inf, D - 1), (-inf, 7), (nan, slice(None)), (-inf, slice(None))]):
        for b in range(B):
            n, h = (5 * i + b) % N, (3 * i + 1) % (g * Hkv)
            q[b, n, h, at] = value
            bad[b, n, h] = True
    q[:, N - 1, 0, 3] = nan
    bad[:, N - 1, 0] = True
    blind = torch.zeros_like(bad)
    for b in range(B):
        blind[b, N - 1] = starts[b] == 0
    got, bad, blind = run(q), bad.cuda(), blind.cuda()
    assert got[bad & ~blind].isnan().all()
    assert torch.equal(got[~bad], want[~bad]) and (got[blind] == 0).all()


def test_rows_that_are_not_computed_are_zero_in_outputs_a_call_makes(nv):
    """Refused sequences and tokens, without counts and without an output of the caller's."""
    q = torch.randn(2, 4, 4, 128, device="cuda").bfloat16()
    x = torch.randn(2, 4, 1, 128, device="cuda").bfloat16()
    k, v = (nv.KVPlane.allocate(2, 1, 64, 128) for _ in range(2))
    sc, tab = torch.tensor([0.01], device="cuda"), make_rope(64, 128).cuda()

    def after_junk(call, dtype=torch.bfloat16):
        junk = [torch.full((2, 4, 4, 128), float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        return call()
    st = status()
    for dtype in (torch.bfloat16, torch.float32):
        got = after_junk(lambda: nv.nvfp4_tree_attention(q, k, v, sc, sc, i32([61, 0]), out_dtype=dtype, status=st), dtype)
        assert st.item() == nv.NVFP4_ERR_CAPACITY and (got == 0).all()          # (the cache holds zeros)
    st = status()
    got = after_junk(lambda: nv.nvfp4_qk_norm_rope_append(q, x, x, i32([0, 61]), sc, sc, k, v, rope_table=tab, status=st))
    assert st.item() == nv.NVFP4_ERR_CAPACITY and (got[1] == 0).all() and (got[0] != 0).any()
    st = status()
    got = after_junk(lambda: nv.nvfp4_qk_norm_rope_append(q, x, x, i32([0, 0]), sc, sc, k, v, rope_table=tab, status=st,
                                                          positions=i32([[0, 1, 64, 2], [0, 1, 2, 3]])))
    assert st.item() == nv.NVFP4_ERR_INVALID_ARG and (got[0, 2] == 0).all() and (got[0, 3] != 0).any()
    st = status()
    got = after_junk(lambda: nv.nvfp4_qk_norm_rope_append(q, x, x, i32([0, 0]), sc * 0, sc, k, v, status=st))
    assert st.item() == nv.NVFP4_ERR_NONFINITE and (got == 0).all()


def test_nothing_to_do_is_no_call(nv):
    """No tokens, no nodes: nothing is written, new_lens neither."""
    k, v = (nv.KVPlane.allocate(2, 1, 64, 128) for _ in range(2))
    q = torch.zeros(2, 0, 4, 128, device="cuda").bfloat16()
    x = torch.zeros(2, 0, 1, 128, device="cuda").bfloat16()
    sc, st, lens = torch.tensor([0.01], device="cuda"), status(), i32([-5, -5])
    assert nv.nvfp4_qk_norm_rope_append(q, x, x, i32([3, 4]), sc, sc, k, v, new_lens=lens, status=st).shape == q.shape
    assert nv.nvfp4_tree_attention(q, k, v, sc, sc, i32([3, 4]), status=st).shape == q.shape
    nv.nvfp4_kv_commit_path([k, v], i32([3, 4]), torch.zeros(2, 0, dtype=torch.int32, device="cuda"), i32([0, 0]),
                            new_lens=lens, status=st)
    assert lens.tolist() == [-5, -5] and st.item() == 0 and not k.codes.any()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,starts,kind,paged", [
    (1, 1024, 2, 1, 128, [300], "tree", False), (2, 1000, 1, 1, 64, [0, 77], "chain", True),
    (1, 513, 6, 2, 128, [1], "star", True), (1, 5, 128, 1, 128, [400], "tree", False),
    (2, 3, 256, 2, 64, [1000, 0], "tree", True), (2, 11, 96, 1, 128, [260, 3000], "tree", False),
    (1, 1, 128, 1, 128, [700], "chain", False), (1, 1, 127, 1, 64, [129], "chain", False)])
def test_tree_attention_to_its_limits(nv, B, N, Hq, Hkv, D, starts, kind, paged, bf16):
    """1,024 nodes; 128 query heads of one KV head."""
    run_tree(nv, B, N, Hq, Hkv, D, starts, kind, bf16, paged=paged, seed=N + Hq)


def test_tree_attention_masks_of_many_nodes(nv):
    rng = np.random.default_rng(8)
    m = rng.random((2, 700, 700)) < 0.02
    m[0, 13] = m[1, 699] = False
    m[1, 5] = True
    run_tree(nv, 2, 700, 2, 1, 64, [0, 45], bf16=True, masks=m, counts=[700, 650])


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("N,kind", [(257, "chain"), (1024, "chain"), (1024, "tree"), (300, "star"), (1024, "star")])
def test_verify_to_its_limit(nv, N, kind, draft):
    """Paths and rejections of hundreds of nodes."""
    p, d, tok, par, ua, us = make_verify(3, N, 700, kind, N, sharp=1.0)
    ua[0] = 0.0                                            # every node that may be: the longest path
    ua[1] = 1.0 - 2.0 ** -24                               # hardly any: all children of the root
    st, n_acc = check_verify(nv, p, d if draft else None, tok, par, ua, us, counts=[N, N, N - 1], shared=kind != "tree")
    assert st == 0 and (kind != "chain" or n_acc[0] == N)


@pytest.mark.parametrize("D,Hkv,paged", [(128, 2, False), (64, 1, True), (64, 70, False)])
def test_commit_of_a_thousand_nodes(nv, D, Hkv, paged):
    rng = np.random.default_rng(Hkv)
    B, N, S, L = 5, 1024, 2048, 2
    codes = torch.from_numpy(rng.integers(0, 256, (L, B, Hkv, S, D // 2), dtype=np.uint8))
    scales = torch.from_numpy(rng.integers(0, 256, (L, B, Hkv, S, D // 16), dtype=np.uint8))
    start, n_acc = [0, S - N, 1000, 3, 77], [N, 700, 257, 0, 256]
    path = np.full((B, N), -1, np.int32)
    for b in range(B):
        path[b, :n_acc[b]] = np.sort(rng.choice(N, n_acc[b], replace=False))
    want_c, want_s = codes.clone(), scales.clone()
    for b in range(B):
        src = start[b] + torch.from_numpy(path[b, :n_acc[b]].astype(np.int64))
        want_c[:, b, :, start[b]:start[b] + n_acc[b]] = codes[:, b][:, :, src]
        want_s[:, b, :, start[b]:start[b] + n_acc[b]] = scales[:, b][:, :, src]
    lens, st, table = i32([-1] * B), status(), None
    if paged:
        table = block_table(B, S // 128, 3)
        lay = lambda t: torch.stack([to_pages([x], table, 128)[0] for x in t])
        codes, scales, want_c, want_s = lay(codes), lay(scales), lay(want_c), lay(want_s)
        table = table.cuda()
    c, s = codes.cuda(), scales.cuda()
    planes = [nv.PagedKVPlane(c[i], s[i], table) if paged else nv.KVPlane(c[i], s[i]) for i in range(L)]
    call = nv.nvfp4_kv_commit_path_paged if paged else nv.nvfp4_kv_commit_path
    call(planes, i32(start), dev(path), i32(n_acc), new_lens=lens, status=st)
    assert torch.equal(c.cpu(), want_c) and torch.equal(s.cpu(), want_s)
    assert lens.tolist() == [a + n for a, n in zip(start, n_acc)] and st.item() == 0


@pytest.mark.parametrize("Hq,Hkv,n,paged", [(128, 1, 3, False), (96, 1, 70, True), (1, 130, 2, False)])
def test_norm_rope_append_head_counts(nv, Hq, Hkv, n, paged):
    run_append(nv, 2, n, Hq, Hkv, 128, 128, "bf16", False, True, True, True, paged, seed=Hq)
    run_append(nv, 2, n, Hq, Hkv, 64, 32, "f32", True, True, False, False, paged, seed=Hq)


def test_tree_attention_over_its_own_queries(nv):
    """bf16 outputs may take the queries' place: a unit reads its rows before it writes them."""
    for B, N, Hq, Hkv, D, S in ((1, 4, 8, 2, 128, 60), (3, 40, 12, 4, 64, 3000), (2, 64, 8, 2, 128, 9000)):
        c, s = synthetic.random_planes(4, B, Hkv, (S + N + 15) // 16 * 16, D, max_scale_byte=0x50)
        k, v = nv.KVPlane(c.cuda(), s.cuda()), nv.KVPlane(c.flip(2).contiguous().cuda(), s.cuda())
        q, sc = torch.randn(B, N, Hq, D, device="cuda").bfloat16(), torch.tensor([0.01], device="cuda")
        want = nv.nvfp4_tree_attention(q, k, v, sc, sc, i32([S] * B), out_dtype=torch.bfloat16)
        for _ in range(5):
            x = q.clone()
            assert nv.nvfp4_tree_attention(x, k, v, sc, sc, i32([S] * B), out=x) is x
            assert torch.equal(x, want)


def test_tree_attention_beside_other_calls(nv):
    """Two streams' tree attention with workspaces of their own, decode attention and
    verification at the same time."""
    c, s = synthetic.random_planes(6, 4, 4, 4096, 128, max_scale_byte=0x50)
    k, v = nv.KVPlane(c.cuda(), s.cuda()), nv.KVPlane(c.flip(2).contiguous().cuda(), s.cuda())
    sc = torch.tensor([0.01], device="cuda")
    ver = [dev(t) for t in make_verify(8, 6, 20000, "tree", 3)]
    jobs = []
    for N, Hq, start in ((8, 16, 4000), (40, 32, 3000)):
        q, st = torch.randn(4, N, Hq, 128, device="cuda").bfloat16(), i32([start, 17, start - 99, 0])
        ws = torch.empty(nv.nvfp4_tree_attention_workspace(4, N, Hq, 4, 128), dtype=torch.uint8, device="cuda")
        jobs.append(lambda q=q, st=st, ws=ws: nv.nvfp4_tree_attention(q, k, v, sc, sc, st, workspace=ws))
    qd, lens = torch.randn(4, 16, 128, device="cuda").bfloat16(), i32([4096, 5, 2000, 900])
    jobs.append(lambda: nv.nvfp4_decode_attention(qd, k, v, sc, sc, lens))
    jobs.append(lambda: torch.stack([nv.nvfp4_verify_drafts(*ver)[i].flatten()[:8] for i in range(3)]))
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(20):
        for j, st, g in zip(jobs, streams, got):
            with torch.cuda.stream(st):
                g.append(j())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, w) for x in g)


FIRST_CALL = """
import torch
import bit_decode_attention_b200 as nv
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
torch.manual_seed(1)
k, v = (nv.KVPlane.allocate(1, 2, 256, 128) for _ in range(2))
x = torch.randn(1, 5, 8, 128, device="cuda").bfloat16()
kv = torch.randn(1, 5, 2, 128, device="cuda").bfloat16()
sc, start = torch.tensor([0.004], device="cuda"), i32(100)
p = torch.softmax(torch.randn(1, 5, 1000, device="cuda"), -1)
args = p, p.flip(1).contiguous(), i32(*range(5))[None], i32(-1, 0, 0, 1, 1), p[:, :, 0].contiguous(), p[:, 0, 0].contiguous()
lens = i32(0)


def step():
    q = nv.nvfp4_qk_norm_rope_append(x, kv, kv, start, sc, sc, k, v)
    o = nv.nvfp4_tree_attention(q, k, v, sc, sc, start)
    path, n, token = nv.nvfp4_verify_drafts(*args)
    nv.nvfp4_kv_commit_path([k, v], start, path, n, new_lens=lens)
    return q, o, path, n, token


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (*got, lens, k.codes, v.codes)]
for t in (k.codes, k.scales, v.codes, v.scales, lens):
    t.zero_()
want = (*step(), lens, k.codes, v.codes)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_a_step_captured_before_any_call(nv):
    """The process's first calls are captured ones: kernels are loaded and set up then."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=200,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
