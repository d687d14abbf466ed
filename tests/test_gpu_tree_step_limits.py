"""The tree-step operators on the GPU at the ends of their documented ranges: nodes and
group sizes up to the limits, values that are no numbers, rows that nobody computes."""
import pytest
import torch

import tree_reference as ref
from test_gpu_tree_step import dev, make_verify, status

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
