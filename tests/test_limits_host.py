"""The largest sizes that fit a launch, from the descriptors alone (host only)."""
import ctypes

import permute_grouped_gemm_amd as pgg

FAKE = 0x100000   # never dereferenced: every call is refused before a launch


def test_gate_tokens_fit_a_launch():
    # 4 rows to a workgroup of 256 lanes, fewer than 2^32 lanes
    for tokens, status in (((1 << 26) - 4, pgg.ERR_INVALID_ARG), ((1 << 26) - 3, pgg.ERR_UNSUPPORTED)):
        d = pgg.GateDesc(tokens, 1000, 2, 1.0, 0, 2, 0)
        assert pgg.lib().pgg_moe_gate(ctypes.byref(d), None, None, FAKE, FAKE, FAKE, None) == status
        assert pgg.lib().pgg_moe_gate_grad(ctypes.byref(d), None, FAKE, FAKE, FAKE, None, FAKE, None) == status


def test_adapter_tokens_fit_a_launch():
    # 8 x 512 lanes to 256 tokens, and one workgroup that checks the ids
    for tokens, status in (((1 << 28) - 256, pgg.OK), ((1 << 28) - 255, pgg.ERR_UNSUPPORTED)):
        n, d = ctypes.c_size_t(), pgg.LoraDesc(tokens, 64, 64, 2, 4, 2, 0)
        assert pgg.lib().pgg_lora_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status


def test_the_gated_products_reduction_stays_in_32_bits():
    # the tiles count reduction elements in 32 bits, up to three stages of 64 past the end
    for k, status in (((1 << 31) - 256, pgg.OK), ((1 << 31) - 255, pgg.ERR_UNSUPPORTED)):
        n, d = ctypes.c_size_t(), pgg.GluDesc(1, k, 1, k, 16, 1, 1, 1, 1, 0, 2, 2, 0)
        assert pgg.lib().pgg_moe_glu_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status
