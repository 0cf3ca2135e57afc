"""Descriptor checks of the gate, the gated products and the adapters through
the C ABI (host only: no GPU is touched)."""
import ctypes

import pytest

import permute_grouped_gemm_amd as pgg

F32, F16, BF16 = 0, 1, 2
FAKE = 0x100000   # never dereferenced: every call below is refused before a launch


def _size(query, d):
    n = ctypes.c_size_t()
    return query(ctypes.byref(d), ctypes.byref(n)), n.value


def gate(tokens=4, experts=16, topk=2, scale=1.0, renorm=0, dtype=BF16, reserved=0):
    return pgg.GateDesc(tokens, experts, topk, scale, renorm, dtype, reserved)


def glu(batch=8, topk=2, G=4, K=32, F=16, dtype=BF16, wd=None, act=0, rit=0, x_rows=None, x_cols=None, idx=None,
        cols=None, gl=None):
    return pgg.GluDesc(batch if x_rows is None else x_rows, K if x_cols is None else x_cols, G, K,
                       2 * F if cols is None else cols, batch * topk if idx is None else idx, G if gl is None else gl,
                       batch, topk, rit, dtype, dtype if wd is None else wd, act)


def glu_grad(M=16, D=32, G=4, F=16, dtype=BF16, wd=None, act=0, gl=None, cols=None, reserved=0):
    return pgg.GluGradDesc(M, D, G, F, D if cols is None else cols, G if gl is None else gl, dtype,
                           dtype if wd is None else wd, act, reserved)


def lora(T=8, K=32, N=16, P=3, R=4, dtype=BF16, reserved=0):
    return pgg.LoraDesc(T, K, N, P, R, dtype, reserved)


def test_struct_sizes():
    # as the header lays them out: 64-bit fields first
    assert ctypes.sizeof(pgg.GateDesc) == 40 and ctypes.sizeof(pgg.LoraDesc) == 48
    assert ctypes.sizeof(pgg.GluDesc) == 9 * 8 + 4 * 4 and ctypes.sizeof(pgg.GluGradDesc) == 6 * 8 + 4 * 4


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=0), 1), (dict(experts=0, topk=0), 1), (dict(topk=0), 1), (dict(topk=17), 1), (dict(renorm=2), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(reserved=1), 1), (dict(experts=8193), 2),
    (dict(experts=100, topk=65), 2), (dict(tokens=1 << 26), 2)])
def test_gate_descriptor(bad, status):
    L = pgg.lib()
    d = gate(**bad)
    assert L.pgg_moe_gate(ctypes.byref(d), FAKE, None, FAKE, FAKE, FAKE, None) == status
    assert L.pgg_moe_gate_grad(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == status


def test_gate_pointers():
    L, d, f = pgg.lib(), gate(), gate(dtype=F32)
    assert L.pgg_moe_gate(None, FAKE, None, FAKE, FAKE, FAKE, None) == pgg.ERR_INVALID_ARG
    for i in (0, 2, 3):
        args = [FAKE, None, FAKE, FAKE, FAKE]
        args[i] = None
        assert L.pgg_moe_gate(ctypes.byref(d), *args, None) == pgg.ERR_INVALID_ARG
    for i, off in ((0, 2), (1, 2), (2, 4), (3, 2), (4, 1)):
        args = [FAKE, FAKE, FAKE, FAKE, FAKE]
        args[i] += off
        assert L.pgg_moe_gate(ctypes.byref(f), *args, None) == pgg.ERR_MISALIGNED
    for i in (0, 1, 2, 3, 5):
        args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
        args[i] = None
        assert L.pgg_moe_gate_grad(ctypes.byref(d), *args, None) == pgg.ERR_INVALID_ARG
    for i, off in ((0, 1), (1, 2), (2, 4), (3, 2), (4, 2), (5, 1)):
        args = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
        args[i] += off
        assert L.pgg_moe_gate_grad(ctypes.byref(d), *args, None) == pgg.ERR_MISALIGNED


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), 1), (dict(topk=0), 1), (dict(G=0), 1), (dict(K=0), 1), (dict(F=0), 1), (dict(cols=31), 1),
    (dict(x_rows=7), 1), (dict(x_cols=31), 1), (dict(idx=15), 1), (dict(gl=3), 1), (dict(rit=2), 1), (dict(act=2), 1),
    (dict(act=-1), 1), (dict(wd=F16), 1), (dict(dtype=5), 1), (dict(batch=1 << 30, topk=2), 2)])
def test_glu_descriptor(bad, status):
    assert _size(pgg.lib().pgg_moe_glu_workspace_size, glu(**bad))[0] == status


@pytest.mark.parametrize("bad,status", [
    (dict(M=0), 1), (dict(D=0), 1), (dict(G=0), 1), (dict(F=0), 1), (dict(cols=31), 1), (dict(gl=5), 1),
    (dict(act=7), 1), (dict(wd=F32), 1), (dict(dtype=9), 1), (dict(reserved=1), 1), (dict(M=1 << 31), 2),
    (dict(F=1 << 30), 2)])
def test_glu_grad_descriptor(bad, status):
    assert _size(pgg.lib().pgg_moe_glu_grad_workspace_size, glu_grad(**bad))[0] == status


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(P=0), 1), (dict(R=0), 1), (dict(dtype=3), 1),
    (dict(reserved=2), 1), (dict(R=1025), 2), (dict(T=1 << 31), 2), (dict(K=1 << 31), 2), (dict(P=1 << 31), 2)])
def test_lora_descriptor(bad, status):
    assert _size(pgg.lib().pgg_lora_workspace_size, lora(**bad))[0] == status


def test_workspace_and_pointer_refusals():
    L = pgg.lib()
    for query, call, d, n_args, optional in (
            (L.pgg_moe_glu_workspace_size, L.pgg_moe_glu, glu(), 6, (5,)),
            (L.pgg_moe_glu_grad_workspace_size, L.pgg_moe_glu_grad, glu_grad(), 6, (5,)),
            (L.pgg_lora_workspace_size, L.pgg_lora_fwd, lora(), 7, ())):
        st, need = _size(query, d)
        assert st == pgg.OK and need > 0
        assert query(ctypes.byref(d), None) == pgg.ERR_INVALID_ARG
        args = [FAKE] * n_args
        for i in range(n_args):
            if i not in optional:
                assert call(ctypes.byref(d), *args[:i], None, *args[i + 1:], FAKE, need, None) == pgg.ERR_INVALID_ARG
            assert call(ctypes.byref(d), *args[:i], FAKE + 1, *args[i + 1:], FAKE, need, None) == pgg.ERR_MISALIGNED
        assert call(ctypes.byref(d), *args, None, need, None) == pgg.ERR_INVALID_ARG
        assert call(ctypes.byref(d), *args, FAKE, need - 1, None) == pgg.ERR_WORKSPACE_TOO_SMALL
        assert call(ctypes.byref(d), *args, FAKE + 128, need, None) == pgg.ERR_MISALIGNED


def test_workspaces_stay_small():
    # tables only where the tiles fill the chip; split partials bounded where they do not
    M, G = 110592, 60
    st, n = _size(pgg.lib().pgg_moe_glu_workspace_size, glu(batch=13824, topk=8, G=G, K=7168, F=1024))
    assert st == pgg.OK and n <= 2 * 4 * M + 8 * (G + 1) + 16 * (M // 256 + G + 1) + 8 * 512
    st, n = _size(pgg.lib().pgg_moe_glu_grad_workspace_size, glu_grad(M=M, D=7168, G=G, F=2048))
    assert st == pgg.OK and n <= 8 * (G + 1) + 16 * (M // 256 + G + 1) + 8 * 512
    st, n = _size(pgg.lib().pgg_lora_workspace_size, lora(T=13824, K=7168, N=2048, P=60, R=16))
    assert st == pgg.OK and n <= 4 * 13824 * 16 + 4 * 512
    for T in (1, 16, 64):
        st, n = _size(pgg.lib().pgg_lora_workspace_size, lora(T=T, K=7168, N=4096, P=60, R=16))
        assert st == pgg.OK and n <= 4 * T * 16 + 64 * 4 * T * 4096 + 4 * 512


def test_planning_random_shapes():
    # any valid shape gets a workspace or a refusal, whatever its sizes
    import random
    r = random.Random(5)
    spread = lambda hi: int(2 ** r.uniform(0, hi))  # noqa: E731
    for _ in range(3000):
        dt = r.randint(0, 2)
        topk = r.randint(1, 8)
        for query, d in ((pgg.lib().pgg_moe_glu_workspace_size, glu(batch=spread(22), topk=topk, G=spread(16), K=spread(18),
                                                                    F=spread(18), dtype=dt)),
                         (pgg.lib().pgg_moe_glu_grad_workspace_size, glu_grad(M=spread(25), D=spread(18), G=spread(16),
                                                                              F=spread(18), dtype=dt)),
                         (pgg.lib().pgg_lora_workspace_size, lora(T=spread(24), K=spread(18), N=spread(18), P=spread(12),
                                                                  R=spread(10), dtype=dt))):
            st, n = _size(query, d)
            assert st in (pgg.OK, pgg.ERR_UNSUPPORTED) and (st != pgg.OK or n >= 512)
