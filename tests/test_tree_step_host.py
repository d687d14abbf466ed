"""Host-side checks of the tree-step entry points: every call below is refused,
or is a no-op, before it reaches the GPU."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import tree_reference as ref
from bit_decode_attention_b200 import _native
from bit_decode_attention_b200 import build as native_build

INVALID, UNSUP, WS = _native.NVFP4_ERR_INVALID_ARG, _native.NVFP4_ERR_UNSUPPORTED, _native.NVFP4_ERR_WORKSPACE
DEV = ctypes.c_void_p(256)      # never dereferenced
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return _native.lib()


def plane(B=2, H=2, S=256, D=128, codes=256, scales=512):
    return _native.KVPlaneStruct(codes, scales, B, H, S, D)


def paged(codes=256, scales=512, table=1024, pages=4, H=2, T=128, D=128, B=2, M=3):
    return _native.PagedPlaneStruct(codes, scales, table, pages, H, T, D, B, M)


def norm_rope(lib, k=None, v=None, pg=False, **kw):
    a = dict(xq=DEV, xk=DEV, xv=DEV, dt=0, n=1, hq=4, sq=0, sk=0, sv=0, wq=DEV, wk=DEV, eps=1e-6, table=DEV, P=64,
             R=128, il=0, pos=None, start=DEV, valid=None, lens=None, stk=DEV, stv=DEV, out=DEV)
    a.update(kw)
    k = k or (paged() if pg else plane())
    v = v or (paged() if pg else plane())
    f = lib.nvfp4_qk_norm_rope_append_paged if pg else lib.nvfp4_qk_norm_rope_append
    return f(a["xq"], a["xk"], a["xv"], a["dt"], a["n"], a["hq"], a["sq"], a["sk"], a["sv"], a["wq"], a["wk"],
             ctypes.c_float(a["eps"]), a["table"], a["P"], a["R"], a["il"], a["pos"], a["start"], a["valid"], a["lens"],
             a["stk"], a["stv"], ctypes.byref(k), ctypes.byref(v), a["out"], None, None)


def test_norm_rope_append_refusals(lib):
    for pg in (False, True):
        for bad in (dict(dt=7), dict(n=-1), dict(hq=0), dict(stk=None), dict(stv=None), dict(start=None),
                    dict(lens=DEV), dict(eps=float("nan")), dict(eps=float("inf")), dict(R=0), dict(R=24),
                    dict(R=144), dict(P=0), dict(table=None), dict(table=ODD), dict(xq=None), dict(xq=ODD),
                    dict(xk=ODD), dict(xv=None), dict(out=None), dict(out=ODD), dict(wq=ODD), dict(wk=ODD),
                    dict(sq=508), dict(sq=516), dict(sk=260), dict(sv=8), dict(sk=-256),
                    dict(valid=DEV, lens=DEV, start=ODD)):
            assert norm_rope(lib, pg=pg, **bad) == INVALID, bad
        assert norm_rope(lib, pg=pg, n=1 << 30) == UNSUP
        assert norm_rope(lib, pg=pg, n=0) == 0
    assert norm_rope(lib, v=plane(S=128)) == INVALID
    assert norm_rope(lib, k=plane(D=96), v=plane(D=96)) == INVALID
    assert norm_rope(lib, k=plane(B=0), v=plane(B=0)) == 0
    assert norm_rope(lib, pg=True, v=paged(table=2048)) == INVALID     # K and V tables differ
    assert norm_rope(lib, pg=True, k=paged(T=96), v=paged(T=96)) == INVALID


def tree(lib, k=None, v=None, pg=False, **kw):
    a = dict(q=DEV, dt=0, N=4, hq=4, stk=DEV, stv=DEV, start=DEV, nodes=None, mask=None, stride=0, scale=0.0, out=DEV,
             odt=1, ws=DEV, nb=1 << 40)
    a.update(kw)
    k = k or (paged() if pg else plane())
    v = v or (paged() if pg else plane())
    f = lib.nvfp4_tree_attention_paged if pg else lib.nvfp4_tree_attention
    return f(a["q"], a["dt"], a["N"], a["hq"], ctypes.byref(k), ctypes.byref(v), a["stk"], a["stv"], a["start"],
             a["nodes"], a["mask"], a["stride"], ctypes.c_float(a["scale"]), a["out"], a["odt"], a["ws"], a["nb"],
             None, None)


def test_tree_attention_refusals(lib):
    for pg in (False, True):
        for bad in (dict(dt=7), dict(odt=7), dict(N=-1), dict(hq=3), dict(hq=0), dict(stk=None), dict(stv=None),
                    dict(start=None), dict(scale=-1.0), dict(scale=float("nan")), dict(q=None), dict(q=ODD),
                    dict(out=None), dict(out=ODD), dict(mask=DEV, stride=3), dict(mask=DEV, stride=-4)):
            assert tree(lib, pg=pg, **bad) == INVALID, bad
        for bad in (dict(dt=1), dict(N=1025), dict(hq=2 * 129)):
            assert tree(lib, pg=pg, **bad) == UNSUP, bad
        for bad in (dict(ws=None), dict(ws=ODD), dict(nb=16)):
            assert tree(lib, pg=pg, **bad) == WS, bad
        assert tree(lib, pg=pg, N=0) == 0
    assert tree(lib, v=plane(S=128)) == INVALID
    assert tree(lib, k=plane(B=0), v=plane(B=0)) == 0
    # 2^9 sequences x 2^10 KV heads x 2^14 tiles of 128 tokens: past 31 bits
    big = plane(B=512, H=1 << 10, S=1 << 21)
    assert tree(lib, k=big, v=big, hq=1 << 10) == UNSUP
    need = lib.nvfp4_tree_attention_workspace(2, 4, 4, 2, 128)
    assert need > 0 and tree(lib, nb=need - 1) == WS
    for shape in ((2, 4, 3, 2, 128), (2, 4, 4, 2, 96), (2, 1025, 4, 2, 128), (2, 4, 258, 2, 128), (-1, 4, 4, 2, 128)):
        assert lib.nvfp4_tree_attention_workspace(*shape) == 0


def test_tree_attention_outputs_over_queries(lib):
    at = lambda i: ctypes.c_void_p((1 << 20) + 16 * i)
    units = 2 * 4 * 4 * 128 * 2 // 16                        # of 16 bytes: bf16 queries of two sequences
    for odt, span in ((0, units), (1, 2 * units)):
        for pg in (False, True):
            for i in (1, units // 2, units - 1, 1 - span):
                assert tree(lib, pg=pg, q=at(0), out=at(i), odt=odt) == INVALID, (odt, i)
    assert tree(lib, q=at(0), out=at(0), odt=1) == INVALID


def test_tree_attention_refuses_tiles_past_32_bits(lib):
    """The last tile of a sequence of more than 2^31 - 128 tokens ends past 31 bits."""
    most = 2 ** 31 - 128
    for S, want in ((most, WS), (most + 16, UNSUP), (most + 112, UNSUP)):
        pl = plane(B=1, H=1, S=S)
        assert tree(lib, k=pl, v=pl, hq=1, N=1, ws=None) == want
    pl = paged(T=128, M=most // 128, B=1)
    assert tree(lib, pg=True, k=pl, v=pl, ws=None, N=1, hq=2) == WS


def test_verify_refusals(lib):
    def call(p=DEV, d=DEV, dt=1, B=2, N=4, V=100, tok=DEV, par=DEV, sh=1, ua=DEV, us=DEV, path=DEV, na=DEV, nx=DEV):
        return lib.nvfp4_verify_drafts(p, d, dt, B, N, V, tok, par, sh, ua, us, None, path, na, nx, None, None)
    for bad in (dict(dt=7), dict(B=-1), dict(N=0), dict(V=0), dict(p=None), dict(tok=None), dict(par=None),
                dict(ua=None), dict(us=None), dict(path=None), dict(na=None), dict(nx=None),
                dict(p=ctypes.c_void_p(258)), dict(d=ctypes.c_void_p(258)), dict(dt=0, p=ctypes.c_void_p(257))):
        assert call(**bad) == INVALID, bad
    assert call(N=1025) == UNSUP
    assert call(B=(1 << 24) + 1) == UNSUP
    assert call(B=0) == 0


def test_commit_refusals(lib):
    def call(planes, n=None, N=4, start=DEV, path=DEV, na=ODD, lens=None, pg=False):
        kind = _native.PagedPlaneStruct if pg else _native.KVPlaneStruct
        arr = (kind * max(1, len(planes)))(*planes)
        f = lib.nvfp4_kv_commit_path_paged if pg else lib.nvfp4_kv_commit_path
        return f(arr, len(planes) if n is None else n, N, start, path, na, lens, None, None)
    for pg, one, others in ((False, plane(), (plane(S=128), plane(H=4), plane(D=64), plane(B=3), plane(codes=257))),
                            (True, paged(), (paged(table=2048), paged(T=256), paged(M=2), paged(pages=0)))):
        for bad in (dict(start=None), dict(path=None), dict(na=None), dict(lens=DEV), dict(lens=ODD), dict(N=-1),
                    dict(n=-1)):
            assert call([one], pg=pg, **bad) == INVALID, bad
        for o in others:
            assert call([one, o], pg=pg) == INVALID
        assert call([one], pg=pg, N=1025) == UNSUP
        assert call([one], pg=pg, N=0) == 0
        assert call([], pg=pg) == 0
    assert call([plane(B=0)]) == 0


def test_commit_refuses_planes_that_share_memory(lib):
    """A launch moves its planes at the same time: one given twice (layers that share a
    cache), or a part of another, would be moved by two blocks at once."""
    def call(planes, pg=False):
        kind = _native.PagedPlaneStruct if pg else _native.KVPlaneStruct
        f = lib.nvfp4_kv_commit_path_paged if pg else lib.nvfp4_kv_commit_path
        # d_new_lens aliasing d_start_pos is refused as well; N = 0 ends the accepted calls early
        return f((kind * len(planes))(*planes), len(planes), 0, DEV, DEV, DEV, None, None, None)
    code, scale = 2 * 2 * 256 * 64, 2 * 2 * 256 * 8          # bytes of plane()
    c0, s0 = 1 << 20, 1 << 30
    at = lambda i, j: plane(codes=c0 + i * code, scales=s0 + j * scale)
    far = [at(i, i) for i in range(300)]
    assert call(far[:2]) == 0 and call(far[::-1]) == 0 and call(far[1:150] + far[:1] + far[200:]) == 0
    for planes in ([at(0, 0), at(0, 0)], [at(0, 0), at(0, 1)], [at(0, 0), at(1, 0)],
                   [at(0, 0), plane(codes=c0 + code - 16, scales=s0 + 9 * scale)],
                   [at(1, 1), plane(codes=c0, scales=s0 + scale + 16)],
                   far + far[7:8], far[9:10] + far[:20], far[::-1] + [far[150]]):
        assert call(planes) == INVALID
    pages = 4 * 2 * 128
    pool = lambda i, j: paged(codes=c0 + i * pages * 64, scales=s0 + j * pages * 8)
    assert call([pool(0, 0), pool(1, 1), pool(2, 5)], True) == 0
    for planes in ([pool(0, 0), pool(0, 1)], [pool(0, 0), pool(3, 1), pool(2, 0)]):
        assert call(planes, True) == INVALID


def test_append_refuses_planes_that_share_memory(lib):
    c, s = 2 * 2 * 256 * 64, 2 * 2 * 256 * 8                 # bytes of plane()
    k = plane(codes=1 << 20, scales=1 << 30)
    for codes, scales in ((1 << 20, 1 << 29), (1 << 25, 1 << 30), ((1 << 20) + c - 16, 1 << 29), (1 << 25, (1 << 30) - s + 16)):
        assert norm_rope(lib, k=k, v=plane(codes=codes, scales=scales)) == INVALID
        assert norm_rope(lib, k=plane(codes=codes, scales=scales), v=k) == INVALID
    k = paged(codes=1 << 20, scales=1 << 30)
    assert norm_rope(lib, pg=True, k=k, v=paged(codes=1 << 20, scales=1 << 29)) == INVALID
    assert norm_rope(lib, pg=True, k=k, v=paged(codes=1 << 25, scales=(1 << 30) + 4 * 2 * 128 * 8 - 16)) == INVALID


def test_outputs_over_inputs_are_refused(lib):
    """Whole numbers that a call writes, over ones that its other blocks may still read."""
    at = lambda i: ctypes.c_void_p(1 << 20 | 4 * i)
    for pg in (False, True):
        # B = 2, n = 3: positions 10 .. 15, starts 20, 21, counts 30, 31
        a = dict(n=3, P=1 << 20, pos=at(10), start=at(20), valid=at(30), pg=pg)
        for i in (9, 10, 12, 15, 19, 20, 21, 29, 31):
            assert norm_rope(lib, lens=at(i), **a) == INVALID, i
        for i in (8, 16, 18, 22, 28, 32):                    # apart: the next check is reached
            assert norm_rope(lib, lens=at(i), **dict(a, n=1 << 30, pos=None)) == UNSUP, i

    def commit(lens, pg):
        one = paged() if pg else plane()
        f = lib.nvfp4_kv_commit_path_paged if pg else lib.nvfp4_kv_commit_path
        return f(ctypes.byref(one), 1, 3, at(20), at(10), at(30), at(lens), None, None)
    for pg in (False, True):
        for i in (9, 10, 15, 19, 21, 29, 31):
            assert commit(i, pg) == INVALID, i

    def verify(**kw):
        b = dict(tok=at(10), par=at(20), sh=0, ua=at(30), us=at(40), nodes=at(50), path=at(100), na=at(110), nx=at(120), N=3)
        b.update(kw)
        return lib.nvfp4_verify_drafts(DEV, DEV, 1, 2, b["N"], 100, b["tok"], b["par"], b["sh"], b["ua"], b["us"],
                                       b["nodes"], b["path"], b["na"], b["nx"], None, None)
    for i in (5, 10, 15, 16, 20, 25, 30, 35, 39, 41, 46, 50, 51):
        assert verify(path=at(i)) == INVALID, i
    for name in ("na", "nx"):
        for i in (9, 15, 20, 25, 29, 35, 39, 41, 99, 100, 105):
            assert verify(**{name: at(i)}) == INVALID, (name, i)
    assert verify(na=at(119)) == INVALID
    # parents of one tree for all sequences: N of them
    assert verify(path=at(22), sh=1) == INVALID


def test_commit_of_no_nodes_needs_no_path(lib):
    for pg, one in ((False, plane()), (True, paged())):
        f = lib.nvfp4_kv_commit_path_paged if pg else lib.nvfp4_kv_commit_path
        call = lambda n, N: f(ctypes.byref(one), n, N, DEV, None, DEV, None, None, None)
        assert call(1, 0) == 0 and call(0, 0) == 0 and call(1, 1) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes(lib, monkeypatch):
    import bit_decode_attention_b200 as nv
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pl = nv.KVPlane(torch.zeros(1, 1, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16, 8, dtype=torch.uint8))
    x = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16)
    one = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_qk_norm_rope_append(x, x, x, i32(1), one, one, pl, pl)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_tree_attention(x, pl, pl, one, one, i32(1))
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_verify_drafts(torch.zeros(1, 2, 8), None, i32(1, 2), i32(2), torch.zeros(1, 2), one)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_kv_commit_path([pl], i32(1), i32(1, 2), i32(1))
    with pytest.raises(TypeError, match="PagedKVPlane"):
        nv.nvfp4_tree_attention_paged(x, pl, pl, one, one, i32(1))
    with pytest.raises(ValueError, match="at least one"):
        nv.KVPlaneList([])


def binding_append(nv, xq, xk, xv, B, H, D=64, eps=float("nan"), interleaved=False):
    """The binding's checks of an append, on host tensors (device -1); eps NaN is refused by
    the library, before any launch: a call that passes the binding returns INVALID."""
    pl = nv.KVPlane(torch.zeros(B, H, 16, D // 2, dtype=torch.uint8), torch.zeros(B, H, 16, D // 16, dtype=torch.uint8))
    one, start = torch.ones(1), torch.zeros(B, dtype=torch.int32)
    out = torch.empty(xq.shape, dtype=xq.dtype)
    return _native.binding().qk_norm_rope_append(-1, 0, False, xq, xk, xv, start, one, one, pl, pl, None, None, eps, None,
                                                 interleaved, None, None, out, None, None)


@pytest.mark.parametrize("B,n,from_shape", [(2, 3, (1, 1)), (2, 1, (1, 1)), (1, 3, (1, 1)), (2, 3, (1, 3)), (2, 3, (2, 1))])
def test_binding_refuses_broadcast_inputs(lib, B, n, from_shape):
    """Memory that holds fewer rows than the shape says (a step of 0 between tokens)."""
    import bit_decode_attention_b200 as nv
    full = torch.zeros(B, n, 2, 64)
    few = torch.zeros(*from_shape, 2, 64).expand(B, n, 2, 64)
    assert binding_append(nv, full, full, full, B, 2) == INVALID
    for at in range(3):
        x = [full] * 3
        x[at] = few
        with pytest.raises(ValueError, match="evenly spaced"):
            binding_append(nv, *x, B, 2)
    # steps below a token's row, without being 0
    over = torch.zeros(2 * 64 + 16 * (B * n - 1) + 64)
    with pytest.raises(ValueError, match="evenly spaced"):
        binding_append(nv, over.as_strided((B, n, 2, 64), (16 * n, 16, 64, 1)), full, full, B, 2)


def test_binding_takes_rows_of_one_token_and_packed_rows(lib):
    import bit_decode_attention_b200 as nv
    one = torch.zeros(64).expand(1, 1, 1, 64)
    assert binding_append(nv, one, one, one, 1, 1) == INVALID
    packed = torch.zeros(2, 3, 4, 64)
    q, k, v = packed[:, :, :2], packed[:, :, 2:3], packed[:, :, 3:]
    assert binding_append(nv, q, k, v, 2, 1) == INVALID
    empty = torch.zeros(2, 0, 1, 64)
    assert binding_append(nv, empty, empty, empty, 2, 1) == INVALID


def test_binding_passes_on_a_failing_truth_value(lib):
    """`interleaved` without a truth value: its own error, and no call."""
    import bit_decode_attention_b200 as nv
    x = torch.zeros(1, 2, 1, 64)
    with pytest.raises(RuntimeError, match="ambiguous"):
        binding_append(nv, x, x, x, 1, 1, interleaved=torch.zeros(2))
    assert binding_append(nv, x, x, x, 1, 1, interleaved=torch.ones(1)) == INVALID


def test_plane_list_keeps_what_its_addresses_name(lib, monkeypatch):
    """The structs are laid out once: planes that a caller adds to the list later, or tensors
    replaced in one, must not change what the call reads or free what it points at."""
    import gc
    import weakref
    import bit_decode_attention_b200 as nv

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0

    real, seen = _native.binding(), []

    class Binding:
        @staticmethod
        def planes(device, paged, planes):
            return real.planes(-1, paged, planes)

        @staticmethod
        def commit_path(device, stream, paged, address, count, *rest):
            seen.append((address, count))
            return 0

    monkeypatch.setattr(_native, "binding", lambda: Binding)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    new = lambda: nv.KVPlane(torch.zeros(1, 1, 16, 64, dtype=torch.uint8).as_subclass(OnDevice),
                             torch.zeros(1, 1, 16, 8, dtype=torch.uint8).as_subclass(OnDevice))
    mine = [new(), new()]
    planes = nv.KVPlaneList(mine)
    codes = weakref.ref(mine[0].codes)
    mine.append(new())
    try:
        planes.planes.append(new())
    except AttributeError:
        pass                                               # not a list any more
    assert len(planes) == 2
    nv.nvfp4_kv_commit_path(planes, None, None, None)
    assert seen == [(planes.address, 2)]
    mine[0].codes = new().codes
    gc.collect()
    assert codes() is not None                             # the structs still name this memory


def test_reference_forms_agree_with_closed_forms():
    # the references the GPU tests compare with, on cases worked by hand
    m = ref.ancestors(ref.parents_of("star", 4))
    assert m.sum() == 7 and m[:, 0].all()
    assert ref.mask_words(m).flatten().tolist() == [1, 3, 5, 9]
    q = np.zeros((2, 1, 64))
    kv = np.ones((1, 5, 64))
    vv = np.arange(5.0)[None, :, None] * np.ones((1, 5, 64))
    out, _, _, _ = ref.tree_attention(q, kv, vv, 3, 2, np.array([[True, False], [False, True]]))
    assert np.allclose(out[0], (0 + 1 + 2 + 3) / 4) and np.allclose(out[1], (0 + 1 + 2 + 4) / 4)
    # one token drafted with certainty: accepted with probability p(x); the rest is p without x
    p = np.array([[0.5, 0.25, 0.25], [0.0, 0.0, 1.0]])
    assert ref.verify(p, None, [0, 0], [-1, 0], [0, 0.49], 0.0, 2) == ([0, 1], 2)
    assert ref.verify(p, None, [0, 0], [-1, 0], [0, 0.5], 0.5, 2) == ([0], 2)
    assert ref.verify(p, None, [0, 0], [-1, 0], [0, 0.5], 0.49, 2) == ([0], 1)
    d = np.array([[0.25, 0.75, 0.0], [0, 0, 1]])
    assert ref.verify(p, d, [0, 1], [-1, 0], [0, 0.4], 0.49, 2) == ([0], 0)
    y, _ = ref.norm_rope(np.array([3.0, 0, 4.0, 0] + [0.0] * 12), None, 0.0, np.array([0.0] * 8 + [1.0] * 8), True)
    assert np.allclose(y[:4], [0, 3 / np.sqrt(25 / 16), 0, 4 / np.sqrt(25 / 16)])


def test_tree_attention_kernels_fit_their_register_split(tmp_path):
    """No stack frame or spill, and as many registers at launch as the warpgroups' shares
    add up to: a larger sum would wait for registers that nobody gives back."""
    src = os.path.join(native_build.CSRC, "nvfp4kv_tree_attention_tc.cu")
    cmd = [native_build.nvcc(), *[f for f in native_build.NVCC_FLAGS if f != "-shared"], "-c", "-Xptxas", "-v",
           "-I", native_build.INCLUDE, "-o", str(tmp_path / "tree.o"), src]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    except FileNotFoundError:
        pytest.skip("nvcc not available")
    assert r.returncode == 0, r.stderr[-2000:]
    found = re.findall(r"Compiling entry function '[^']*tree_attention_tc_kernelINS0_3CfgILi(\d+)ELi(\d)E[^']*'.*?\n"
                       r".*?(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads.*?"
                       r"Used (\d+) registers", r.stderr, flags=re.S)
    assert len(found) == 8
    for _, rb, stack, stores, loads, regs in found:
        assert (stack, stores, loads) == ("0", "0", "0")
        threads, shares = (896, 256 * 112 + 128 * 56 + 512 * 56) if rb == "1" else (640, 256 * 136 + 128 * 64 + 256 * 72)
        assert shares <= threads * int(regs) <= 65536
