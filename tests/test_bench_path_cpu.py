"""The path whose name bench.py puts on a workload's kernels is the one that the layer call takes."""
import ctypes

import pytest

import bench
import indirect_expert_matmul_amd as moe
import synth

FAKE = 0x10000  # sizes only


def _workspace(cfg, T, wtype, path, aq):
    w = lambda n, r, c: moe.c_moe_weights(wtype, FAKE, FAKE, n, r, c)
    g = w(cfg.n_experts, cfg.n_ff, cfg.n_embd)
    sg = ctypes.byref(w(cfg.n_shared, cfg.n_ff, cfg.n_embd)) if cfg.n_shared else None
    opt = moe._options(path, act_quant=aq)
    return moe.lib.moe_ffn_fused_workspace_size(ctypes.byref(g), sg, moe.MOE_BF16, T, cfg.n_used, ctypes.byref(opt))


@pytest.mark.parametrize("T,n_embd,n_ff,S", [(1, 2880, 2880, 0), (1, 2880, 96, 0), (1, 96, 2880, 0), (16, 256, 128, 3),
                                             (16, 256, 128, 5), (13, 256, 128, 5), (17, 256, 128, 0), (1, 128, 96, 1)])
def test_mxfp4_activations(T, n_embd, n_ff, S):
    cfg = synth.Config("x", "ffn", 32, 4, T, n_embd, n_ff, n_shared=S, wtype="mxfp4")
    got = bench.ffn_path(moe, cfg, T, 4, moe.MOE_MXFP4, moe.PATH_AUTO, 2)
    forced = _workspace(cfg, T, moe.MOE_MXFP4, {4: moe.PATH_GEMM, 5: moe.PATH_GEMV}[got], 2)
    assert forced == _workspace(cfg, T, moe.MOE_MXFP4, moe.PATH_AUTO, 2) > 0
    other = _workspace(cfg, T, moe.MOE_MXFP4, {5: moe.PATH_GEMM, 4: moe.PATH_GEMV}[got], 2)
    assert other != forced                       # 0: the other path cannot run it


def test_other_workloads_keep_theirs():
    for name in ("lite", "dec1", "dec8", "dec1x", "dec8x", "ppx"):
        cfg = synth.CONFIGS[name]
        wtype = moe.MOE_MXFP4 if cfg.wtype == "mxfp4" else moe.MOE_Q8_0
        want = moe.moe_select_path_typed(cfg.n_tokens, cfg.n_used, cfg.n_experts, max(cfg.n_embd, cfg.n_ff), wtype)
        assert bench.ffn_path(moe, cfg, cfg.n_tokens, cfg.n_used, wtype, moe.PATH_AUTO, 0) == want
