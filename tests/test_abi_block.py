"""Descriptor and pointer checks of the grouped gate, the 4-bit products and the
combination through the C ABI (host only: no GPU is touched)."""
import ctypes

import pytest

import permute_grouped_gemm_amd as pgg

F32, F16, BF16 = 0, 1, 2
FAKE = 0x100000   # never dereferenced: every call below is refused before a launch


def _size(query, d):
    n = ctypes.c_size_t()
    return query(ctypes.byref(d), ctypes.byref(n)), n.value


def gate(T=4, E=16, k=2, groups=4, kept=2, scale=1.0, score=0, renorm=1, dtype=BF16):
    return pgg.GateGroupedDesc(T, E, k, groups, kept, scale, score, renorm, dtype)


def w4(G=3, K=64, N=32, gs=32, dtype=BF16, zeros=0, gated=0, reserved=0):
    return pgg.W4Desc(G, K, N, gs, dtype, zeros, gated, reserved)


def moe_w4(batch=5, topk=2, x_rows=None, x_cols=None, idx=None, gl=None, rit=0, act=0, **w):
    d = w4(**w)
    return pgg.MoeW4Desc(d, batch if x_rows is None else x_rows, d.rows if x_cols is None else x_cols,
                         batch * topk if idx is None else idx, d.groups if gl is None else gl, batch, topk, rit, act)


def combine(batch=4, topk=2, H=64, alpha=1.0, eps=1e-6, rit=0, dtype=BF16):
    return pgg.CombineDesc(batch, topk, H, alpha, eps, rit, dtype)


def test_struct_sizes():
    assert ctypes.sizeof(pgg.GateGroupedDesc) == 5 * 8 + 4 * 4 and ctypes.sizeof(pgg.W4Desc) == 4 * 8 + 4 * 4
    assert ctypes.sizeof(pgg.MoeW4Desc) == 48 + 6 * 8 + 2 * 4 and ctypes.sizeof(pgg.CombineDesc) == 3 * 8 + 4 * 4
    assert ctypes.sizeof(pgg.CombineGradArgs) == 15 * 8


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(kept=0), 1), (dict(kept=5), 1),
    (dict(groups=3), 1), (dict(groups=32), 1), (dict(k=9), 1), (dict(kept=1, k=5), 1), (dict(score=2), 1),
    (dict(score=-1), 1), (dict(renorm=2), 1), (dict(dtype=3), 1), (dict(E=8196), 2),
    (dict(E=256, groups=2, kept=2, k=65), 2), (dict(E=130, groups=65, kept=65), 2), (dict(T=(1 << 26) - 3), 2)])
def test_gate_descriptor(bad, status):
    L, d = pgg.lib(), gate(**bad)
    assert L.pgg_moe_gate_grouped(ctypes.byref(d), FAKE, None, FAKE, FAKE, None) == status
    assert L.pgg_moe_gate_grouped_grad(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, None) == status


def test_gate_pointers():
    L, f = pgg.lib(), gate(dtype=F32)
    assert L.pgg_moe_gate_grouped(None, FAKE, None, FAKE, FAKE, None) == pgg.ERR_INVALID_ARG
    for call, optional, misaligned in ((L.pgg_moe_gate_grouped, (1,), ((0, 2), (1, 2), (2, 4), (3, 2))),
                                       (L.pgg_moe_gate_grouped_grad, (), ((0, 2), (1, 4), (2, 2), (3, 1)))):
        for i in range(4):
            if i not in optional:
                args = [FAKE] * 4
                args[i] = None
                assert call(ctypes.byref(f), *args, None) == pgg.ERR_INVALID_ARG
        for i, off in misaligned:
            args = [FAKE] * 4
            args[i] += off
            assert call(ctypes.byref(f), *args, None) == pgg.ERR_MISALIGNED


@pytest.mark.parametrize("bad,status", [
    (dict(G=0), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(gs=0), 1), (dict(gs=16), 1), (dict(gs=96), 1),
    (dict(gs=200), 1), (dict(dtype=3), 1), (dict(zeros=2), 1), (dict(gated=2), 1), (dict(gated=1, N=31), 1),
    (dict(reserved=1), 1), (dict(G=1 << 30), 2), (dict(K=1 << 16, N=1 << 16), 2), (dict(K=1 << 31), 2)])
def test_w4_descriptor(bad, status):
    L, d = pgg.lib(), w4(**bad)
    assert _size(L.pgg_w4_pack_size, d)[0] == status
    assert L.pgg_w4_pack(ctypes.byref(d), FAKE, FAKE, None, FAKE, None) == status
    m = moe_w4(**bad)
    assert _size(L.pgg_moe_w4_workspace_size, m)[0] == status


def test_w4_pack_pointers():
    L, d, z = pgg.lib(), w4(), w4(zeros=1)
    st, n = _size(L.pgg_w4_pack_size, d)
    assert st == pgg.OK and n >= 3 * 64 * 32 // 2
    assert L.pgg_w4_pack_size(ctypes.byref(d), None) == pgg.ERR_INVALID_ARG
    for i in (0, 1, 3):
        args = [FAKE, FAKE, None, FAKE]
        args[i] = None
        assert L.pgg_w4_pack(ctypes.byref(d), *args, None) == pgg.ERR_INVALID_ARG
    assert L.pgg_w4_pack(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, None) == pgg.ERR_INVALID_ARG
    assert L.pgg_w4_pack(ctypes.byref(z), FAKE, FAKE, None, FAKE, None) == pgg.ERR_INVALID_ARG
    assert L.pgg_w4_pack(ctypes.byref(d), FAKE, FAKE + 1, None, FAKE, None) == pgg.ERR_MISALIGNED
    assert L.pgg_w4_pack(ctypes.byref(d), FAKE, FAKE, None, FAKE + 128, None) == pgg.ERR_MISALIGNED


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), 1), (dict(topk=0), 1), (dict(x_rows=4), 1), (dict(x_cols=63), 1), (dict(idx=9), 1),
    (dict(idx=0), 1), (dict(gl=2), 1), (dict(rit=2), 1), (dict(act=2), 1), (dict(batch=1 << 30), 2),
    (dict(batch=1 << 27, N=2048), 2)])
def test_moe_w4_descriptor(bad, status):
    L, d = pgg.lib(), moe_w4(**bad)
    assert _size(L.pgg_moe_w4_workspace_size, d)[0] == status
    assert L.pgg_moe_fwd_w4(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == status


def test_moe_w4_pointers():
    L = pgg.lib()
    for call, d in ((L.pgg_moe_fwd_w4, moe_w4()), (L.pgg_moe_glu_w4, moe_w4(gated=1))):
        st, need = _size(L.pgg_moe_w4_workspace_size, d)
        assert st == pgg.OK and need >= 512
        args = [FAKE] * 5
        for i in range(5):
            assert call(ctypes.byref(d), *args[:i], None, *args[i + 1:], FAKE, need, None) == pgg.ERR_INVALID_ARG
            assert call(ctypes.byref(d), *args[:i], FAKE + 1, *args[i + 1:], FAKE, need, None) == pgg.ERR_MISALIGNED
        assert call(ctypes.byref(d), *args, None, need, None) == pgg.ERR_INVALID_ARG
        assert call(ctypes.byref(d), *args, FAKE, need - 1, None) == pgg.ERR_WORKSPACE_TOO_SMALL
        assert call(ctypes.byref(d), *args, FAKE + 128, need, None) == pgg.ERR_MISALIGNED
    # weights of the other kind; an index where none was announced
    assert L.pgg_moe_glu_w4(ctypes.byref(moe_w4()), *args, FAKE, 1 << 30, None) == pgg.ERR_INVALID_ARG
    assert L.pgg_moe_fwd_w4(ctypes.byref(moe_w4(gated=1)), *args, FAKE, 1 << 30, None) == pgg.ERR_INVALID_ARG
    ordered = moe_w4(topk=1, idx=0)
    assert L.pgg_moe_fwd_w4(ctypes.byref(ordered), *args, FAKE, 1 << 30, None) == pgg.ERR_INVALID_ARG


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), 1), (dict(topk=0), 1), (dict(H=0), 1), (dict(rit=2), 1), (dict(dtype=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(H=16385), 2), (dict(batch=1 << 30), 2)])
def test_combine_descriptor(bad, status):
    L, d = pgg.lib(), combine(**bad)
    assert _size(L.pgg_moe_combine_workspace_size, d)[0] == status
    assert _size(L.pgg_moe_combine_grad_workspace_size, d)[0] == status
    assert L.pgg_moe_combine(ctypes.byref(d), *[FAKE] * 9, FAKE, 1 << 40, None) == status


def test_combine_pointers():
    L, d = pgg.lib(), combine()
    st, need = _size(L.pgg_moe_combine_workspace_size, d)
    assert st == pgg.OK
    args = [FAKE] * 9
    for i in range(9):
        refused = L.pgg_moe_combine(ctypes.byref(d), *args[:i], None, *args[i + 1:], FAKE, need - 1, None)
        # post_weight and gate may be missing; next_weight and normed only together
        assert refused == (pgg.ERR_WORKSPACE_TOO_SMALL if i in (4, 5) else pgg.ERR_INVALID_ARG)
        assert L.pgg_moe_combine(ctypes.byref(d), *args[:i], FAKE + 1, *args[i + 1:], FAKE, need, None) == \
            pgg.ERR_MISALIGNED
    assert L.pgg_moe_combine(ctypes.byref(d), *args, None, need, None) == pgg.ERR_INVALID_ARG
    assert L.pgg_moe_combine(ctypes.byref(d), *args, FAKE, need - 1, None) == pgg.ERR_WORKSPACE_TOO_SMALL
    assert L.pgg_moe_combine(ctypes.byref(d), *args, FAKE + 64, need, None) == pgg.ERR_MISALIGNED


def test_combine_grad_pointers():
    L, d = pgg.lib(), combine()
    st, need = _size(L.pgg_moe_combine_grad_workspace_size, d)
    assert st == pgg.OK and need >= 2 * 4 * 64 * 4
    names = [n for n, _ in pgg.CombineGradArgs._fields_]

    def call(ws=FAKE, size=need, **change):
        a = pgg.CombineGradArgs(**{**{n: FAKE for n in names}, **change})
        return L.pgg_moe_combine_grad(ctypes.byref(d), ctypes.byref(a), ws, size, None)

    for n in names:
        # of each optional pair one alone is refused
        assert call(**{n: None}) == pgg.ERR_INVALID_ARG, n
        assert call(**{n: FAKE + 1}) == pgg.ERR_MISALIGNED, n
    for pair in (("gate", "grad_gate"), ("post_weight", "grad_post_weight"),
                 ("next_weight", "grad_next_weight", "grad_normed")):
        assert call(size=need - 1, **{n: None for n in pair}) == pgg.ERR_WORKSPACE_TOO_SMALL
    assert call(ws=None) == pgg.ERR_INVALID_ARG and call(size=need - 1) == pgg.ERR_WORKSPACE_TOO_SMALL
    assert call(ws=FAKE + 128) == pgg.ERR_MISALIGNED
    assert L.pgg_moe_combine_grad(ctypes.byref(d), None, FAKE, need, None) == pgg.ERR_INVALID_ARG


def test_planning_random_shapes():
    # any valid shape gets a workspace or a refusal, whatever its sizes
    import random
    r = random.Random(6)
    spread = lambda hi: int(2 ** r.uniform(0, hi))  # noqa: E731
    for _ in range(3000):
        dt, topk = r.randint(0, 2), r.randint(1, 8)
        d = moe_w4(batch=spread(24), topk=topk, G=spread(14), K=spread(17), N=2 * spread(16), gs=r.choice((32, 64, 128)),
                   dtype=dt, gated=r.randint(0, 1), zeros=r.randint(0, 1))
        c = combine(batch=spread(27), topk=topk, H=spread(15), dtype=dt, rit=r.randint(0, 1))
        for query, desc in ((pgg.lib().pgg_moe_w4_workspace_size, d), (pgg.lib().pgg_w4_pack_size, d.weight),
                            (pgg.lib().pgg_moe_combine_workspace_size, c),
                            (pgg.lib().pgg_moe_combine_grad_workspace_size, c)):
            st, n = _size(query, desc)
            assert st in (pgg.OK, pgg.ERR_UNSUPPORTED) and (st != pgg.OK or n >= 512)


def test_workspaces_stay_small():
    M = 16384   # tables, and partial results only where the reduction is split
    st, n = _size(pgg.lib().pgg_moe_w4_workspace_size, moe_w4(batch=2048, topk=8, G=16, K=7168, N=4096, gs=128, gated=1))
    assert st == pgg.OK and n <= 2 * 4 * M + 17 * 8 + 16 * (M + 16) + 8 * 512 + 4 * 2048 * 7168 // 32
    st, n = _size(pgg.lib().pgg_moe_combine_grad_workspace_size, combine(batch=13824, topk=8, H=7168))
    assert st == pgg.OK and n <= 2 * 4 * 110592 + 2 * 4 * 4096 * 7168


def test_sizes_that_fit_a_launch():
    L = pgg.lib()
    # 4 rows to a workgroup of 256 lanes at most 1024 experts, a row to a wave above
    for tokens, status in (((1 << 26) - 4, pgg.ERR_INVALID_ARG), ((1 << 26) - 3, pgg.ERR_UNSUPPORTED)):
        d = gate(T=tokens, E=1000, groups=1, kept=1)
        assert L.pgg_moe_gate_grouped(ctypes.byref(d), None, None, FAKE, FAKE, None) == status
        assert L.pgg_moe_gate_grouped_grad(ctypes.byref(d), None, FAKE, FAKE, FAKE, None) == status
    # 256 lanes to 16 rows (fp32) and 256 columns
    for rows, status in ((16 * ((1 << 24) - 2), pgg.OK), (16 * ((1 << 24) - 1), pgg.ERR_UNSUPPORTED)):
        d = moe_w4(batch=rows, topk=1, idx=0, G=1, K=32, N=64, dtype=F32)
        assert _size(L.pgg_moe_w4_workspace_size, d)[0] == status
    # a workgroup of 64 lanes to a token
    for batch, status in (((1 << 26) - 1025, pgg.OK), ((1 << 26) - 1024, pgg.ERR_UNSUPPORTED)):
        assert _size(L.pgg_moe_combine_workspace_size, combine(batch=batch, topk=1, H=8))[0] == status
