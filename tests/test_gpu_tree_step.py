"""The tree-step operators on the GPU against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import oracle
import synthetic
import tree_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_decode_attention_b200 as nv
    return nv


def dev(a, dtype=None):
    t = torch.as_tensor(a)
    return (t if dtype is None else t.to(dtype)).contiguous().cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def np8(t):
    return t.cpu().numpy()


def block_table(B, pages_each, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(B * pages_each, generator=g).to(torch.int32).reshape(B, pages_each)


def to_pages(planes, table, T):
    """[B][H][M * T][X] -> pool [B * M][H][T][X] laid out by the table."""
    B, M = table.shape
    out = []
    for p in planes:
        H, X = p.shape[1], p.shape[3]
        pool = torch.zeros(B * M, H, T, X, dtype=p.dtype)
        pool[table.long().flatten()] = p.reshape(B, H, M, T, X).permute(0, 2, 1, 3, 4).reshape(B * M, H, T, X)
        out.append(pool)
    return out


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,Hkv,N,n_planes", [(128, 8, 6, 4), (64, 1, 1, 1), (64, 3, 40, 2), (128, 60, 17, 2),
                                              (128, 2, 9, 67)])
@pytest.mark.parametrize("paged", [False, True])
def test_commit_moves_the_path(nv, D, Hkv, N, n_planes, paged):
    rng = np.random.default_rng(N * 7 + Hkv)
    B, S = 5, 256
    codes = torch.from_numpy(rng.integers(0, 256, (n_planes, B, Hkv, S, D // 2), dtype=np.uint8))
    scales = torch.from_numpy(rng.integers(0, 256, (n_planes, B, Hkv, S, D // 16), dtype=np.uint8))
    start = [0, S - N, 120, 3, 77]
    n_acc = [N, min(2, N), 0, 1, (N + 1) // 2]
    path = np.full((B, N), -7, np.int32)
    for b in range(B):
        path[b, :n_acc[b]] = np.sort(rng.choice(N, n_acc[b], replace=False))
    want_c, want_s = codes.clone(), scales.clone()
    for b in range(B):
        src = start[b] + torch.from_numpy(path[b, :n_acc[b]].astype(np.int64))
        want_c[:, b, :, start[b]:start[b] + n_acc[b]] = codes[:, b][:, :, src]
        want_s[:, b, :, start[b]:start[b] + n_acc[b]] = scales[:, b][:, :, src]
    lens, st = i32([-1] * B), status()
    if paged:
        table = block_table(B, S // 128, 3)
        lay = lambda t: torch.stack([to_pages([x], table, 128)[0] for x in t])
        codes, scales, want_c, want_s = lay(codes), lay(scales), lay(want_c), lay(want_s)
        table = table.cuda()
    c, s = codes.cuda(), scales.cuda()
    planes = [nv.PagedKVPlane(c[i], s[i], table) if paged else nv.KVPlane(c[i], s[i]) for i in range(n_planes)]
    call = nv.nvfp4_kv_commit_path_paged if paged else nv.nvfp4_kv_commit_path
    call(planes, i32(start), dev(path), i32(n_acc), new_lens=lens, status=st)
    assert torch.equal(c.cpu(), want_c) and torch.equal(s.cpu(), want_s)
    assert lens.tolist() == [a + n for a, n in zip(start, n_acc)] and st.item() == 0


@pytest.mark.parametrize("start,n_acc,path,code", [
    (0, 2, [1, 1, 2], 1), (0, 2, [2, 1, 0], 1), (0, 2, [0, 3, 0], 1), (0, 2, [-1, 1, 2], 1), (0, 4, [0, 1, 2], 1),
    (0, -1, [0, 1, 2], 1), (-1, 1, [0, 1, 2], 1), (14, 3, [0, 1, 2], 3), (14, 2, [0, 2, 2], 3), (2147483647, 1, [0, 1, 2], 3)])
def test_commit_skips_bad_sequences(nv, start, n_acc, path, code):
    c = torch.randint(0, 256, (2, 1, 16, 64), dtype=torch.uint8, device="cuda")
    s = torch.randint(0, 256, (2, 1, 16, 8), dtype=torch.uint8, device="cuda")
    c0, s0, lens, st = c.clone(), s.clone(), i32([-5, -5]), status()
    nv.nvfp4_kv_commit_path([nv.KVPlane(c, s)], i32([start, 0]), i32([path, [0, 2, 9]]), i32([n_acc, 2]), new_lens=lens,
                            status=st)
    assert st.item() == code and lens.tolist() == [-5, 2]
    assert torch.equal(c[0], c0[0]) and torch.equal(s[0], s0[0])
    assert torch.equal(c[1, 0, 1], c0[1, 0, 2]) and torch.equal(s[1, 0, 1], s0[1, 0, 2])


def test_commit_bad_page_is_reported(nv):
    c = torch.randint(0, 256, (2, 1, 128, 64), dtype=torch.uint8, device="cuda")
    s = torch.randint(0, 256, (2, 1, 128, 8), dtype=torch.uint8, device="cuda")
    c0, st = c.clone(), status()
    pl = nv.PagedKVPlane(c, s, i32([[0, 5]]))
    # node 1 (slot 127) moves within page 0; node 2 (slot 128) lies in a page outside the pool
    nv.nvfp4_kv_commit_path_paged([pl], i32([125]), i32([[0, 2, 3, -1]]), i32([3]), status=st)
    assert st.item() == nv.NVFP4_ERR_INVALID_ARG
    assert torch.equal(c[0, 0, 126], c0[0, 0, 127]) and torch.equal(c[0, 0, 127], c0[0, 0, 127])
    assert torch.equal(c[1], c0[1])


# ---------------------------------------------------------------------------
# verify
# ---------------------------------------------------------------------------
def make_verify(B, N, V, kind, seed, dtype=torch.float32, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    base = torch.randn(B, N, V, generator=g) * sharp
    p = torch.softmax(base, -1).to(dtype)
    d = torch.softmax(base + 0.8 * torch.randn(B, N, V, generator=g), -1).to(dtype)
    par = ref.parents_of(kind, N)
    tok = torch.zeros(B, N, dtype=torch.int64)
    for i in range(1, N):
        tok[:, i] = torch.multinomial(d[:, par[i]].float(), 1, generator=g)[:, 0]
    ua, us = torch.rand(B, N, generator=g), torch.rand(B, generator=g)
    return p, d, tok.to(torch.int32), torch.tensor(par, dtype=torch.int32), ua, us


def check_verify(nv, p, d, tok, par, ua, us, counts=None, shared=True):
    B, N, V = p.shape
    st = status()
    parents = par if shared else par[None].repeat(B, 1)
    out = nv.nvfp4_verify_drafts(dev(p), None if d is None else dev(d), dev(tok), dev(parents), dev(ua), dev(us),
                                 n_nodes=None if counts is None else i32(counts), status=st)
    path, n_acc, nxt = (t.cpu().numpy() for t in out)
    for b in range(B):
        n = N if counts is None else counts[b]
        if n == 0:
            assert path[b].tolist() == [-1] * N and n_acc[b] == 0 and nxt[b] == -1
            continue
        want, token = ref.verify(p[b].double().numpy(), None if d is None else d[b].double().numpy(), tok[b].tolist(),
                                 par.tolist(), ua[b].double().numpy(), float(us[b]), n)
        assert path[b].tolist() == want + [-1] * (N - len(want))
        assert n_acc[b] == len(want) and nxt[b] == token
    return st.item(), n_acc


@pytest.mark.parametrize("B,N,V,kind", [(3, 1, 7, "chain"), (4, 5, 1000, "chain"), (2, 3, 1, "star"),
                                        (16, 12, 4099, "tree"), (5, 9, 32000, "star"), (2, 4, 131073, "tree"),
                                        (1, 3, 200064, "star")])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_matches_the_walk(nv, B, N, V, kind, draft, dtype):
    p, d, tok, par, ua, us = make_verify(B, N, V, kind, 11 * N + V, dtype)
    st, _ = check_verify(nv, p, d if draft else None, tok, par, ua, us, shared=N % 2 == 0)
    assert st == 0


def test_verify_many_rejections_and_ragged_counts(nv):
    # a target far from the draft: most children are rejected, some nodes have many
    g = torch.Generator().manual_seed(5)
    B, N, V = 24, 20, 5000
    p = torch.softmax(torch.randn(B, N, V, generator=g) * 3, -1)
    d = torch.softmax(torch.randn(B, N, V, generator=g) * 3, -1)
    par = torch.tensor([-1] + [0] * 9 + [1 + i % 9 for i in range(10)], dtype=torch.int32)
    tok = torch.zeros(B, N, dtype=torch.int32)
    for i in range(1, N):
        tok[:, i] = torch.multinomial(d[:, int(par[i])], 1, generator=g)[:, 0].to(torch.int32)
    ua, us = torch.rand(B, N, generator=g), torch.rand(B, generator=g)
    counts = [N, 1, 0, 7] * 6
    for dd in (d, None):
        st, _ = check_verify(nv, p, dd, tok, par, ua, us, counts)
        assert st == 0


def test_verify_edges(nv):
    V = 4096
    p = torch.zeros(6, 3, V)
    d = torch.zeros(6, 3, V)
    p[:, 0, 5] = 1.0
    d[:, 0, 9] = 1.0
    p[:, 1, 7] = 1.0
    p[:, 2, 8] = 1.0
    tok = torch.tensor([[0, 9, 5]] * 6, dtype=torch.int32)
    par = torch.tensor([-1, 0, 0], dtype=torch.int32)
    ua = torch.zeros(6, 3)
    us = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24, 0.0, 0.0, 0.0])
    # sequence 3: draft and target alike -- nothing is left after a forced rejection (u = 1): the weights stay
    d[3, 0] = 0
    d[3, 0, 5] = 1.0
    tok[3] = torch.tensor([0, 5, 5])
    ua[3] = 1.0
    # sequence 4: NaN and negative target entries count as nothing
    p[4, 0, 0], p[4, 0, 1] = float("nan"), -3.0
    # sequence 5: the child is accepted and its row is empty
    tok[5] = torch.tensor([0, 5, 9])
    d[5, 0, 5] = 0.5
    p[5, 1] = 0
    st, n_acc = check_verify(nv, p, d, tok, par, ua, us)
    assert st == nv.NVFP4_ERR_NONFINITE and n_acc.tolist() == [1 + 1, 2, 2, 1, 2, 2]


def test_verify_bad_nodes_are_reported_and_never_accepted(nv):
    p, d, tok, par, ua, us = make_verify(2, 4, 500, "star", 3)
    ua[:] = 0.0                                           # every good node would be accepted
    for bad_tok, bad_par in ((-1, 0), (500, 0), (2 ** 31 - 1, 0), (5, 1), (5, -1), (5, 7)):
        t, q = tok.clone(), par.clone()
        t[:, 1], q[1] = bad_tok, bad_par
        st = status()
        path, n_acc, _ = nv.nvfp4_verify_drafts(dev(p), dev(d), dev(t), dev(q), dev(ua), dev(us), status=st)
        assert st.item() == nv.NVFP4_ERR_INVALID_ARG
        assert path.tolist() == [[0, 2, -1, -1]] * 2 and n_acc.tolist() == [2, 2]
    st = status()
    path = i32([[9] * 4] * 2)
    nv.nvfp4_verify_drafts(dev(p), dev(d), dev(tok), dev(par), dev(ua), dev(us), n_nodes=i32([5, -1]), path=path, status=st)
    assert st.item() == nv.NVFP4_ERR_INVALID_ARG and path.tolist() == [[9] * 4] * 2


# ---------------------------------------------------------------------------
# norm + rotation + append
# ---------------------------------------------------------------------------
def make_rope(P, R, seed=0):
    inv = 10000.0 ** (-np.arange(0, R, 2) / R)
    ang = np.arange(P)[:, None] * inv
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float()


def run_append(nv, B, n, Hq, Hkv, D, R, dtype, interleaved, norm, weights, packed, paged, counts=None, positions=None,
               seed=0, S=256, T=128):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gain = torch.exp(torch.randn(Hq + 2 * Hkv, D, generator=g))
    x = (torch.randn(B, n, Hq + 2 * Hkv, D, generator=g) * gain).to(dt)
    parts = list(x.split([Hq, Hkv, Hkv], 2))
    xd = x.cuda()
    xq, xk, xv = xd.split([Hq, Hkv, Hkv], 2) if packed else (t.contiguous() for t in xd.split([Hq, Hkv, Hkv], 2))
    wq, wk = ((1 + 0.3 * torch.randn(2, D, generator=g)).to(dt) if weights else (None, None))
    start = [(37 * b) % (S - n + 1) for b in range(B)]
    table = make_rope(512, R) if R else None
    sk, sv = torch.tensor([0.0123]), torch.tensor([0.0177])
    M = S // T
    tbl = block_table(B, M, seed) if paged else None
    tbl_d = tbl.cuda() if paged else None
    new = lambda: nv.PagedKVPlane.allocate(B * M, Hkv, T, D, tbl_d) if paged else nv.KVPlane.allocate(B, Hkv, S, D)
    k, v = new(), new()
    for p in (k, v):                                        # what is not written has to stay
        p.codes.fill_(0xA5)
        p.scales.fill_(0x5A)
    dt_out = torch.full((B, n, Hq, D), 3.0, dtype=dt, device="cuda")
    lens, st = i32([-1] * B), status()
    eps = 1e-5 if norm else -1.0
    call = nv.nvfp4_qk_norm_rope_append_paged if paged else nv.nvfp4_qk_norm_rope_append
    q = call(xq, xk, xv, i32(start), sk.cuda(), sv.cuda(), k, v, w_q=None if wq is None else wq.cuda(),
             w_k=None if wk is None else wk.cuda(), eps=eps, rope_table=None if table is None else table.cuda(),
             interleaved=interleaved, positions=None if positions is None else i32(positions),
             n_valid=None if counts is None else i32(counts), q_out=dt_out, new_lens=lens, status=st)
    assert q is dt_out and st.item() == 0
    cnt = counts if counts is not None else [n] * B
    assert lens.tolist() == [s + c for s, c in zip(start, cnt)]
    pos = np.array(positions) if positions is not None else np.array(start)[:, None] + np.arange(n)
    cs = (table.double().numpy()[pos] if R else np.zeros((B, n, 0)))[:, :, None]
    want, err = ref.norm_rope(parts[0].double().numpy(), None if wq is None else wq.double().numpy(), eps, cs, interleaved)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    got = q.double().cpu().numpy()
    kw, ke = ref.norm_rope(parts[1].double().numpy(), None if wk is None else wk.double().numpy(), eps, cs, interleaved)

    def planes(p):
        if not paged:
            return np8(p.codes), np8(p.scales)
        flat = lambda a: a[tbl.long()].permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * T, -1).numpy()
        return flat(p.codes.cpu()), flat(p.scales.cpu())
    (kc, ks), (vc, vs) = planes(k), planes(v)
    oc, os_ = oracle.new_planes(B, Hkv, S, D)
    assert oracle.quantize_append(parts[2].float().numpy(), np.array(start, np.int32), np.float32(0.0177), oc, os_) == 0
    for b in range(B):
        c, a = cnt[b], start[b]
        assert np.all(np.abs(got[b, :c] - want[b, :c]) <= err[b, :c] + half * np.abs(want[b, :c]))
        assert np.all(got[b, c:] == 3.0)
        ref.check_quantized(kc[b, :, a:a + c], ks[b, :, a:a + c], kw[b, :c].transpose(1, 0, 2), ke[b, :c].transpose(1, 0, 2),
                            float(sk.double()))
        assert np.array_equal(vc[b, :, a:a + c], oc[b, :, a:a + c]) and np.array_equal(vs[b, :, a:a + c], os_[b, :, a:a + c])
        for p, f in ((kc, 0xA5), (vc, 0xA5), (ks, 0x5A), (vs, 0x5A)):
            assert np.all(p[b, :, :a] == f) and np.all(p[b, :, a + c:] == f)


@pytest.mark.parametrize("B,n,Hq,Hkv,D,R,dtype,interleaved,norm,weights,packed,paged", [
    (1, 1, 1, 1, 64, 64, "bf16", False, True, True, False, False),
    (2, 3, 8, 2, 128, 128, "bf16", False, True, True, True, False),
    (2, 3, 8, 2, 128, 128, "f32", True, True, True, True, True),
    (3, 5, 6, 3, 64, 64, "f32", False, True, False, False, True),
    (2, 4, 5, 1, 128, 64, "bf16", False, True, True, True, False),
    (2, 4, 7, 1, 128, 16, "f32", False, False, False, False, False),
    (2, 4, 12, 4, 128, 48, "bf16", True, True, True, False, True),
    (1, 9, 3, 3, 128, 112, "bf16", False, False, False, True, False),
    (2, 2, 4, 2, 64, 48, "bf16", False, True, True, True, True),
    (2, 2, 4, 2, 64, 0, "bf16", False, True, True, True, False),
    (1, 200, 96, 8, 128, 128, "bf16", True, True, True, True, False),
    (40, 8, 32, 8, 128, 64, "bf16", False, True, True, True, True),
])
def test_norm_rope_append(nv, B, n, Hq, Hkv, D, R, dtype, interleaved, norm, weights, packed, paged):
    run_append(nv, B, n, Hq, Hkv, D, R, dtype, interleaved, norm, weights, packed, paged, seed=B + n)


def test_norm_rope_append_padding_and_positions(nv):
    run_append(nv, 4, 5, 4, 2, 128, 128, "bf16", False, True, True, True, False, counts=[5, 0, 1, 3],
               positions=[[511, 0, 7, 7, 2]] * 4)
    run_append(nv, 4, 5, 4, 2, 64, 32, "f32", False, True, True, False, True, counts=[5, 0, 1, 3],
               positions=[[511, 0, 7, 7, 2]] * 4)


def test_append_without_norm_and_rotation_is_quantize_append(nv):
    # the same codes and scale bytes, special blocks and NaN / infinities included
    rows = torch.cat([synthetic.special_blocks(128), synthetic.nonfinite_blocks(128)])
    n = rows.shape[0]
    for dt in (torch.float32, torch.bfloat16):
        x = rows.to(dt).cuda().view(1, n, 1, 128).contiguous()
        for s in (1.0, 0.01, 1e-30, 3e4):
            sc = torch.tensor([s], device="cuda")
            a = [nv.KVPlane.allocate(1, 1, 16, 128) for _ in range(4)]
            q = nv.nvfp4_qk_norm_rope_append(x, x, x, i32([0]), sc, sc, a[0], a[1], eps=-1.0)
            nv.nvfp4_kv_quantize_append_kv(x, x, i32([0]), sc, sc, a[2], a[3])
            for i in (0, 1):
                assert torch.equal(a[i].codes, a[2].codes) and torch.equal(a[i].scales, a[2].scales)
            nan = x.isnan()                                 # a NaN stays one, its payload is not kept
            assert torch.equal(q.isnan(), nan) and torch.equal(q[~nan], x[~nan])


def test_norm_rope_append_errors(nv):
    x = torch.randn(2, 3, 4, 128, device="cuda").bfloat16()
    tab = make_rope(64, 128).cuda()

    def call(start, valid=None, pos=None, s=0.01, table=None):
        k, v = (nv.KVPlane.allocate(2, 4, 32, 128) for _ in range(2))
        st, q = status(), torch.full_like(x, 3.0)
        sc = torch.tensor([s], device="cuda")
        nv.nvfp4_qk_norm_rope_append(x, x, x, i32(start), sc, torch.tensor([0.01], device="cuda"), k, v, rope_table=tab,
                                     n_valid=None if valid is None else i32(valid),
                                     positions=None if pos is None else i32(pos), q_out=q, status=st)
        return st.item(), q, k
    for start in ([30, 0], [-1, 0], [2 ** 31 - 1, 0]):
        st, q, k = call(start)
        assert st == nv.NVFP4_ERR_CAPACITY and (q[0] == 3).all() and not (q[1] == 3).all()
        assert not k.codes[0].any() and k.codes[1].any()
    for valid in ([4, 3], [-1, 3]):
        st, q, k = call([0, 0], valid)
        assert st == nv.NVFP4_ERR_INVALID_ARG and (q[0] == 3).all() and not k.codes[0].any()
    st, q, k = call([0, 0], pos=[[0, 64, 2], [0, 1, -1]])
    assert st == nv.NVFP4_ERR_INVALID_ARG and (q[0, 1] == 3).all() and (q[1, 2] == 3).all()
    assert not (q[0, 2] == 3).all() and not k.codes[0, :, 1].any() and k.codes[0, :, 2].any()
    for s in (0.0, -1.0, float("inf"), float("nan")):
        st, q, k = call([0, 0], s=s)
        assert st == nv.NVFP4_ERR_NONFINITE and (q == 3).all() and not k.codes.any()
    k, v = (nv.PagedKVPlane.allocate(2, 4, 128, 128, t) for t in [i32([[0], [7]])] for _ in range(2))
    st, sc = status(), torch.tensor([0.01], device="cuda")
    q = nv.nvfp4_qk_norm_rope_append_paged(x, x, x, i32([0, 0]), sc, sc, k, v, rope_table=tab, status=st)
    assert st.item() == nv.NVFP4_ERR_INVALID_ARG and k.codes[0].any() and not k.codes[1].any() and q[1].any()


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------
def run_tree(nv, B, N, Hq, Hkv, D, starts, kind="tree", bf16=True, paged=False, counts=None, scale=0.0, S=None, T=128,
             seed=0, masks=None, sharp=1.0, oracle_seqs=None):
    g = torch.Generator().manual_seed(seed)
    M = -(-(max(starts) + N) // T)
    S = S or (M * T if paged else -(-(max(starts) + N) // 16) * 16)
    x = [torch.randn(B, S, Hkv, D, generator=g) * torch.exp(0.5 * torch.randn(Hkv, D, generator=g)) for _ in range(2)]
    s = [np.float32(float(t.abs().max()) / 2688.0) for t in x]
    planes = []
    for t, st in zip(x, s):
        c, sc = oracle.new_planes(B, Hkv, S, D)
        assert oracle.quantize_append(t.numpy(), np.zeros(B, np.int32), st, c, sc) == 0
        planes += [c, sc]
    q = (torch.randn(B, N, Hq, D, generator=g) * sharp).bfloat16()
    seen = ref.ancestors(ref.parents_of(kind, N)) if masks is None else masks
    mask = None if kind == "chain" and masks is None else dev(ref.mask_words(seen))
    t4 = [torch.from_numpy(p) for p in planes]
    if paged:
        tbl = block_table(B, M, seed)
        t4 = to_pages(t4, tbl, T)
    t4 = [t.cuda() for t in t4]
    mk = (lambda a, b: nv.PagedKVPlane(a, b, tbl_d)) if paged else nv.KVPlane
    tbl_d = tbl.cuda() if paged else None
    k, v = mk(t4[0], t4[1]), mk(t4[2], t4[3])
    out = torch.full((B, N, Hq, D), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    ws = torch.full((nv.nvfp4_tree_attention_workspace(B, N, Hq, Hkv, D),), 0xFF, dtype=torch.uint8, device="cuda")
    st = status()
    call = nv.nvfp4_tree_attention_paged if paged else nv.nvfp4_tree_attention
    args = (q.cuda(), k, v, dev([s[0]]), dev([s[1]]), i32(starts))
    kw = dict(tree_mask=mask, n_nodes=None if counts is None else i32(counts), softmax_scale=scale, workspace=ws, status=st)
    got_t = call(*args, out=out, **kw)
    assert got_t is out and st.item() == 0
    got = out.double().cpu().numpy()
    again = call(*args, out=torch.full_like(out, 7.0), **kw)
    assert torch.equal(again.view(torch.uint8), out.view(torch.uint8))          # the same every time
    kf, vf = ref.fp8_values(planes[0], planes[1], s[0]), ref.fp8_values(planes[2], planes[3], s[1])
    worst = 0.0
    for b in range(B) if oracle_seqs is None else oracle_seqs:
        n = N if counts is None else counts[b]
        sb = seen[b] if seen.ndim == 3 else seen
        want, mag, wk, flat = ref.tree_attention(q[b].double().numpy(), kf[b], vf[b], starts[b], n, sb,
                                           None if scale == 0.0 else scale)
        tol = ref.attention_tolerance(want, mag, wk, flat, starts[b] + n, bf16)
        err = np.abs(got[b, :n] - want)
        assert np.all(err <= tol), (b, err.max(), (err / tol).max())
        assert np.all(got[b, n:] == 7.0)
        worst = max(worst, float((err / tol).max()) if err.size else 0.0)
    return worst


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,starts,kind", [
    (1, 1, 1, 1, 128, [0], "chain"),
    (1, 4, 4, 1, 128, [60], "chain"),
    (1, 5, 2, 2, 64, [127], "tree"),
    (2, 8, 8, 2, 128, [300, 1], "tree"),
    (3, 16, 4, 1, 64, [0, 128, 1000], "star"),
    (2, 33, 8, 2, 128, [130, 700], "tree"),
    (1, 64, 8, 2, 128, [513], "tree"),
    (1, 40, 12, 1, 128, [250], "tree"),
    (2, 70, 8, 1, 64, [400, 31], "tree"),
    (1, 130, 3, 1, 128, [77], "tree"),
    (5, 3, 6, 2, 128, [5, 4000, 129, 640, 2047], "chain"),
])
def test_tree_attention(nv, B, N, Hq, Hkv, D, starts, kind, bf16):
    run_tree(nv, B, N, Hq, Hkv, D, starts, kind, bf16, seed=N + B)


@pytest.mark.parametrize("T,D,N", [(128, 128, 9), (256, 64, 20), (128, 128, 64)])
@pytest.mark.parametrize("bf16", [True, False])
def test_tree_attention_paged(nv, T, D, N, bf16):
    run_tree(nv, 3, N, 8, 2, D, [250, 0, 515], "tree", bf16, paged=True, T=T, seed=T)


def test_tree_attention_ragged_counts_and_padding(nv):
    run_tree(nv, 6, 12, 8, 2, 128, [100, 0, 260, 5, 900, 0], "tree", True, counts=[12, 0, 1, 7, 3, 1])
    run_tree(nv, 4, 40, 8, 1, 64, [100, 0, 260, 900], "tree", False, counts=[40, 17, 3, 0], paged=True)


def test_tree_attention_masks(nv):
    # one mask per sequence; rows that see nothing (start 0), only others, or everything
    rng = np.random.default_rng(2)
    m = rng.random((3, 37, 37)) < 0.3
    m[0, 5] = False
    m[0, 6] = True
    m[1, 0] = False
    m[2, 36] = False
    for bf16 in (True, False):
        run_tree(nv, 3, 37, 4, 1, 128, [0, 0, 90], bf16=bf16, masks=m)


def test_tree_attention_scale_and_sharp_scores(nv):
    run_tree(nv, 2, 6, 8, 2, 128, [700, 40], "tree", False, scale=0.5, sharp=3.0)
    run_tree(nv, 2, 6, 8, 2, 128, [700, 40], "tree", True, scale=0.01)
    run_tree(nv, 1, 20, 16, 1, 128, [3000], "tree", True, sharp=30.0)


def test_tree_attention_large_batch_is_split_into_launches(nv):
    B = 600
    run_tree(nv, B, 2, 2, 1, 64, [(b * 13) % 300 for b in range(B)], "chain", True, oracle_seqs=[0, 1, 300, 511, 512, 599])


def test_tree_attention_long_context(nv):
    run_tree(nv, 1, 24, 12, 1, 128, [20000], "tree", False, seed=4)
    run_tree(nv, 1, 8, 8, 1, 128, [40000], "tree", True, seed=5)


def test_chain_of_one_is_decode_attention(nv):
    # one node without a mask attends as nvfp4_decode_attention does
    for D, paged in ((128, False), (64, True)):
        c, s = synthetic.random_planes(9, 2, 2, 640, D, max_scale_byte=0x50)
        q = torch.randn(2, 1, 8, D).bfloat16().cuda()
        sc = torch.tensor([0.02], device="cuda")
        k, v = nv.KVPlane(c.cuda(), s.cuda()), nv.KVPlane(c.flip(2).contiguous().cuda(), s.flip(2).contiguous().cuda())
        lens = i32([601, 7])
        want = nv.nvfp4_decode_attention(q[:, 0].contiguous(), k, v, sc, sc, lens)
        got = nv.nvfp4_tree_attention(q, k, v, sc, sc, lens - 1)
        err = (got[:, 0] - want).abs().max().item()
        assert err <= 1e-3 * want.abs().max().item()      # decode attention's own three-term weights: 2^-12


def test_tree_attention_errors(nv):
    k, v = (nv.KVPlane.allocate(2, 1, 64, 128) for _ in range(2))
    q = torch.randn(2, 4, 2, 128, device="cuda").bfloat16()
    sc = torch.tensor([0.01], device="cuda")

    def call(start, nodes=None, s=sc):
        st, out = status(), torch.full((2, 4, 2, 128), 7.0, device="cuda")
        nv.nvfp4_tree_attention(q, k, v, s, sc, i32(start), n_nodes=None if nodes is None else i32(nodes), out=out, status=st)
        return st.item(), out
    for start in ([61, 0], [-1, 0], [2 ** 31 - 1, 0]):
        st, out = call(start)
        assert st == nv.NVFP4_ERR_CAPACITY and (out[0] == 7).all() and (out[1] == 0).all()
    for nodes in ([5, 4], [-1, 4]):
        st, out = call([0, 0], nodes)
        assert st == nv.NVFP4_ERR_INVALID_ARG and (out[0] == 7).all() and (out[1] == 0).all()
    assert call([0, 0], s=torch.tensor([0.0], device="cuda"))[0] == nv.NVFP4_ERR_NONFINITE
    pk, pv = (nv.PagedKVPlane.allocate(2, 1, 128, 128, t) for t in [i32([[0], [9]])] for _ in range(2))
    st = status()
    nv.nvfp4_tree_attention_paged(q, pk, pv, sc, sc, i32([0, 0]), status=st)
    assert st.item() == nv.NVFP4_ERR_INVALID_ARG


def test_tree_attention_wait_timeout_reports_and_recovers(nv):
    c, s = synthetic.random_planes(3, 1, 1, 640, 128, max_scale_byte=0x50)
    k, v = nv.KVPlane(c.cuda(), s.cuda()), nv.KVPlane(c.cuda(), s.cuda())
    q, sc = torch.randn(1, 4, 2, 128, device="cuda").bfloat16(), torch.tensor([0.01], device="cuda")
    want = nv.nvfp4_tree_attention(q, k, v, sc, sc, i32([600]))
    try:
        nv.nvfp4_set_wait_limit(0)
        st = status()
        nv.nvfp4_tree_attention(q, k, v, sc, sc, i32([600]), status=st)
        assert st.item() == nv.NVFP4_ERR_TIMEOUT
    finally:
        nv.nvfp4_set_wait_limit(-1)
    st = status()
    got = nv.nvfp4_tree_attention(q, k, v, sc, sc, i32([600]), status=st)
    assert st.item() == 0 and torch.equal(got, want)


# ---------------------------------------------------------------------------
# a whole step, captured and replayed, on another stream
# ---------------------------------------------------------------------------
class Step:
    """Two layers of a model's attention over one cache, for one drafted tree."""

    def __init__(self, nv, seed, stream=None):
        self.nv, self.stream = nv, stream
        B, N, Hq, Hkv, D, V = 3, 7, 8, 2, 128, 1000
        self.dims = B, N, Hq, Hkv, D, V
        g = torch.Generator().manual_seed(seed)
        self.qkv = torch.randn(2, B, N, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
        self.start0 = i32([0, 0, 0])
        self.start = i32([200, 31, 126])
        self.planes = [[nv.KVPlane.allocate(B, Hkv, 256, D) for _ in range(2)] for _ in range(2)]
        past = torch.randn(2, 2, B, 200, Hkv, D, generator=g).bfloat16().cuda()
        self.sc = torch.tensor([0.004], device="cuda")
        for l in range(2):
            for w in range(2):
                nv.nvfp4_kv_quantize_append(past[l, w], self.start0, self.sc, self.planes[l][w])
        self.table = make_rope(512, D).cuda()
        self.w = (1 + 0.1 * torch.randn(2, D, generator=g)).bfloat16().cuda()
        self.par = torch.tensor(ref.parents_of("tree", N), dtype=torch.int32)
        seen = ref.ancestors(self.par.tolist())
        self.mask = dev(ref.mask_words(seen))
        depth = torch.from_numpy(seen.sum(1) - 1).to(torch.int32)
        self.pos = (self.start.cpu()[:, None] + depth).to(torch.int32).cuda()
        p, d, tok, par, ua, us = make_verify(B, N, V, "tree", seed)
        self.ver = [dev(t) for t in (p, d, tok, par, ua, us)]
        self.q = torch.zeros(B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(2, B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(nv.nvfp4_tree_attention_workspace(B, N, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        self.path, self.n_acc, self.next, self.lens = i32([[0] * N] * B), i32([0] * B), i32([0] * B), i32([0] * B)
        self.st = status()
        self.list = nv.KVPlaneList(p for l in self.planes for p in l)

    def run(self):
        nv, (B, N, Hq, Hkv, D, V), st = self.nv, self.dims, self.stream
        for l in range(2):
            xq, xk, xv = self.qkv[l].split([Hq, Hkv, Hkv], 2)
            k, v = self.planes[l]
            nv.nvfp4_qk_norm_rope_append(xq, xk, xv, self.start, self.sc, self.sc, k, v, w_q=self.w[0], w_k=self.w[1],
                                         rope_table=self.table, positions=self.pos, q_out=self.q, status=self.st, stream=st)
            nv.nvfp4_tree_attention(self.q, k, v, self.sc, self.sc, self.start, tree_mask=self.mask, out=self.out[l],
                                    workspace=self.ws, status=self.st, stream=st)
        nv.nvfp4_verify_drafts(*self.ver, path=self.path, n_accepted=self.n_acc, next_token=self.next, status=self.st,
                               stream=st)
        nv.nvfp4_kv_commit_path(self.list, self.start, self.path, self.n_acc, new_lens=self.lens, status=self.st,
                                stream=st)

    def state(self):
        return [t.clone() for t in (self.out, self.path, self.n_acc, self.next, self.lens,
                                    *(x for l in self.planes for p in l for x in (p.codes, p.scales)))]


def test_step_keeps_what_a_model_without_drafts_would_cache(nv):
    """After the step the cache holds the accepted nodes as if they had been
    appended one by one, and a decode over it sees what the last node saw."""
    s = Step(nv, 1)
    s.run()
    torch.cuda.synchronize()
    B, N, Hq, Hkv, D, V = s.dims
    assert s.st.item() == 0
    assert torch.equal(s.lens, s.start + s.n_acc)
    paths = s.path.cpu().numpy()
    for b in range(B):
        n = s.n_acc[b].item()
        assert paths[b, 0] == 0 and all(s.par[paths[b, j]] == paths[b, j - 1] for j in range(1, n))
    # the same cache from plain appends of the accepted nodes
    t = Step(nv, 1)
    for l in range(2):
        for b in range(B):
            keep = s.path[b, :s.n_acc[b].item()].long()
            x = t.qkv[l, b:b + 1][:, keep]
            sub = [nv.KVPlane(p.codes[b:b + 1], p.scales[b:b + 1]) for p in t.planes[l]]
            xq, xk, xv = x.split([Hq, Hkv, Hkv], 2)
            nv.nvfp4_qk_norm_rope_append(xq, xk, xv, t.start[b:b + 1], t.sc, t.sc, *sub, w_q=t.w[0], w_k=t.w[1],
                                         rope_table=t.table)
            L = s.lens[b].item()
            for p, q in zip(s.planes[l], t.planes[l]):
                assert torch.equal(p.codes[b, :, :L], q.codes[b, :, :L])
                assert torch.equal(p.scales[b, :, :L], q.scales[b, :, :L])
            # the last accepted node's attention is a decode over the kept cache
            qn = nv.nvfp4_qk_norm_rope_append(xq, xk, xv, t.start[b:b + 1], t.sc, t.sc, *sub, w_q=t.w[0], w_k=t.w[1],
                                              rope_table=t.table)
            want = nv.nvfp4_decode_attention(qn[:, -1].contiguous(), *sub, t.sc, t.sc, s.lens[b:b + 1].contiguous())
            got = s.out[l, b, keep[-1]].float()
            assert (got - want[0]).abs().max().item() <= 2.0 ** -7 * want.abs().max().item()


def test_step_captured_replayed_and_on_another_stream(nv):
    want = Step(nv, 2)
    want.run()
    torch.cuda.synchronize()
    ref_state = want.state()
    # a stream of its own
    side = torch.cuda.Stream()
    a = Step(nv, 2, stream=side)
    torch.cuda.synchronize()
    a.run()
    side.synchronize()
    for x, y in zip(a.state(), ref_state):
        assert torch.equal(x, y)
    # captured once, replayed on new inputs
    b, c = Step(nv, 2), Step(nv, 3)
    other = Step(nv, 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(b.state(), ref_state):
        assert torch.equal(x, y)
    c.run()
    for mine, new in zip((b.qkv, b.w, *b.ver, *(x for l in b.planes for p in l for x in (p.codes, p.scales))),
                         (other.qkv, other.w, *other.ver, *(x for l in other.planes for p in l for x in (p.codes, p.scales)))):
        mine.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(b.state(), c.state()):
        assert torch.equal(x, y)


def test_outputs_made_by_a_call_belong_to_its_stream(nv):
    """With `stream` given and no outputs or workspace, what the call makes for
    itself is neither filled late by the current stream nor reused by it early."""
    torch.manual_seed(5)
    c, s = synthetic.random_planes(11, 2, 2, 640, 128, max_scale_byte=0x50)
    k, v = nv.KVPlane(c.cuda(), s.cuda()), nv.KVPlane(c.cuda(), s.cuda())
    q, sc = torch.randn(2, 8, 4, 128, device="cuda").bfloat16(), torch.tensor([0.01], device="cuda")
    x = torch.randn(2, 8, 2, 128, device="cuda").bfloat16()
    start, counts = i32([600, 300]), i32([8, 5])
    p = torch.softmax(torch.randn(2, 8, 3000, device="cuda"), -1)
    d = torch.softmax(torch.randn(2, 8, 3000, device="cuda"), -1)
    tok, par = torch.randint(0, 3000, (2, 8), device="cuda", dtype=torch.int32), i32([-1, 0, 0, 1, 1, 2, 2, 3])
    ua, us = torch.rand(2, 8, device="cuda"), torch.rand(2, device="cuda")

    def calls(stream):
        o = nv.nvfp4_tree_attention(q, k, v, sc, sc, start, n_nodes=counts, stream=stream)
        y = nv.nvfp4_qk_norm_rope_append(q, x, x, start, sc, sc, k, v, n_valid=counts, stream=stream)
        return [o, y, *nv.nvfp4_verify_drafts(p, d, tok, par, ua, us, n_nodes=counts, stream=stream)]
    calls(None)                                       # the nodes' own slots hold what each call below appends
    want = calls(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                     # the current stream is late ..
    late = calls(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                 # .. or early
    early = calls(side)
    size = nv.nvfp4_tree_attention_workspace(2, 8, 4, 2, 128)
    junk = [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk
    for got in (late, early):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N,g", [(8, 4), (33, 1), (16, 4), (13, 5), (32, 4), (43, 3), (64, 4), (257, 1)])
def test_tree_attention_row_counts(nv, N, g, D, bf16):
    """Rows 32, 33, 64, 65, 128, 129, 256, 257 of a KV head: where their copies and blocks change."""
    run_tree(nv, 2, N, 2 * g, 2, D, [700, 130], "tree", bf16, seed=N + g)


@pytest.mark.parametrize("D", [128, 64])
def test_tree_attention_long_segments(nv, D):
    """Ranges of more than 32 tiles of one unit (on 148 SMs): the fp32 outputs' sums are
    flushed and joined, next to units that the ranges cut."""
    run_tree(nv, 18, 2, 16, 8, D, [4400 + 7 * b for b in range(18)], "chain", False, seed=3, oracle_seqs=[0, 9, 17])


@pytest.mark.parametrize("B,N,Hq,Hkv,D,S", [(2, 8, 8, 2, 128, 5000), (1, 64, 8, 2, 128, 9000), (3, 40, 12, 4, 64, 3000)])
def test_tree_attention_times_out_anywhere_and_recovers(nv, B, N, Hq, Hkv, D, S):
    """Limits between giving up at once and never: whichever waits run out, the call
    returns, says so, and the next one is right."""
    S16 = (S + N + 15) // 16 * 16
    c, s = synthetic.random_planes(4, B, Hkv, S16, D, max_scale_byte=0x50)
    k, v = nv.KVPlane(c.cuda(), s.cuda()), nv.KVPlane(c.cuda(), s.cuda())
    q, sc = torch.randn(B, N, Hq, D, device="cuda").bfloat16(), torch.tensor([0.01], device="cuda")
    start = i32([S] * B)
    for dtype in (torch.float32, torch.bfloat16):
        want = nv.nvfp4_tree_attention(q, k, v, sc, sc, start, out_dtype=dtype)
        for limit in (0, 1, 0, 2, 3):
            st = status()
            try:
                nv.nvfp4_set_wait_limit(limit)
                got = nv.nvfp4_tree_attention(q, k, v, sc, sc, start, out_dtype=dtype, status=st)
                torch.cuda.synchronize()
            finally:
                nv.nvfp4_set_wait_limit(-1)
            assert st.item() in (0, nv.NVFP4_ERR_TIMEOUT)
            if st.item() == 0:
                assert torch.equal(got, want)
            st = status()
            assert torch.equal(nv.nvfp4_tree_attention(q, k, v, sc, sc, start, out_dtype=dtype, status=st), want)
            assert st.item() == 0
