"""Calls of the training step's operators that their documentation allows and that lie at its edges."""
import numpy as np
import pytest
import torch

from test_step_gpu import BF, F32, adam_tensors, copy_of, e4m3_table, hold_reference, mix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def check_steps(a, b, steps):
    """a: a tensor after `steps` steps of AdamW in 8 bits, betas 0.9 and 0.99, from step 1 on; b: before
    them, with the same gradients. The codes and scales of the definition, each one."""
    f = np.float32
    tab = np.concatenate([e4m3_table(), [np.nan]]).astype(f)
    tab = np.concatenate([tab, -tab])
    n = b["p"].numel()
    g = b["g"].float().cpu().numpy()
    codes = {k: b[k].cpu().numpy() for k in ("m", "v", "m_scale", "v_scale")}
    old = np.seterr(over="ignore", under="ignore")
    for step in range(1, steps + 1):
        sm, sv = (np.repeat(codes[k], 128)[:n] for k in ("m_scale", "v_scale"))
        m, v = tab[codes["m"]] * sm, tab[codes["v"]] * sv
        v = v * v
        m = f(0.9) * m + f(1 - 0.9) * g
        v = f(0.99) * v + f(1 - 0.99) * (g * g)
        root = np.sqrt(v)
        key = mix(np.array([(b["seed"] ^ (step * 0x9E3779B9)) & 0xFFFFFFFF], np.uint32))
        key = mix(key ^ np.arange((n + 127) // 128, dtype=np.uint32))
        place = (np.arange(128, dtype=np.uint64) * 0x9E3779B9).astype(np.uint32)
        r = mix(key[:, None] + place[None, :]).reshape(-1)
        for name, x, r16 in (("m", m, r >> np.uint32(16)), ("v", root, r & np.uint32(0xFFFF))):
            codes[name], codes[name + "_scale"] = hold_reference(x, r16, name == "v")
    np.seterr(**old)
    for name in ("m", "v"):
        assert np.array_equal(a[name + "_scale"].cpu().numpy(), codes[name + "_scale"]), name
        assert np.array_equal(a[name].cpu().numpy() & 127, codes[name] & 127), name
    assert bool(torch.isfinite(a["p"]).all())


def many(large, small):
    """250 tensors, the even ones about twice as large as the odd ones: 2125 whole chunks of 4096
    elements, three or four to each of the kernel's 608 CTAs, which so meet borders of tensors."""
    return [(4096 * (2 + i % 20) + large * i if i % 2 == 0 else 4096 * (1 + i % 10) + small * i)
            for i in range(250)]


@pytest.mark.parametrize("sizes,gtypes", [([5_000_011], [F32]), ([5_000_011], [BF]),
                                          (many(1, 3), [F32, BF]), (many(3, 1), [BF, F32])],
                         ids=["fp32", "bf16", "mostly fp32", "mostly bf16"])
def test_adamw_8_bit_chunk_after_chunk(moe, sizes, gtypes):
    """CTAs that take several chunks, of tensors with gradients of the other type beside: a tensor
    gets the codes of the definition, each of many what it gets alone."""
    A = adam_tensors(sizes, 8, gtypes, seed=5)
    B = copy_of(A)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    plan, state = moe.AdamTensors(A, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    steps = 2 if len(sizes) == 1 else 4
    for _ in range(steps):
        moe.adamw(cfg, plan, state)
    if len(sizes) == 1:
        check_steps(A[0], B[0], steps)
        return
    for i, (a, b) in enumerate(zip(A, B)):
        own, st = moe.AdamTensors([b], state_bits=8), moe.adam_state(0, 0.9, 0.99)
        for _ in range(steps):
            moe.adamw(cfg, own, st)
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            assert torch.equal(a[k], b[k]), (i, k)
        assert b["w"] is None or torch.equal(a["w"], b["w"])
