"""The attention layer of examples/attention_layer.py on the GPU: its decode steps against its
own prompt over the same tokens, and the command itself."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a GPU")
    import gpu_util

    gpu_util.lib_ready()
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_decode_continues_the_prompt(example):
    # prompts of n tokens, then token by token, against prompts of all tokens at once: the same
    # layer but for the cache's e4m3 keys and values (4 significant bits: 2^-4 of each)
    hidden, hq, hk, d, page = 512, 8, 2, 64, 32
    lens, extra = [70, 5], 40
    g = torch.Generator("cuda").manual_seed(3)
    w_qkv = (torch.randn((hq + 2 * hk) * d, hidden, generator=g, device="cuda") * hidden ** -0.5).bfloat16()
    w_out = (torch.randn(hidden, hq * d, generator=g, device="cuda") * (hq * d) ** -0.5).bfloat16()
    rows = [torch.randn(n + extra, hidden, generator=g, device="cuda").bfloat16() for n in lens]
    table = torch.arange(2 * 4, dtype=torch.int32, device="cuda").view(2, 4)
    whole, steps = (example.AttentionLayer(hidden, hq, hk, d, w_qkv, w_out, 512, 8, page) for _ in range(2))
    cu = torch.tensor([0, lens[0] + extra, sum(lens) + 2 * extra], dtype=torch.int32, device="cuda")
    want = whole.prompt(torch.cat(rows), table, cu).float()
    cu0 = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    first = steps.prompt(torch.cat([r[:n] for r, n in zip(rows, lens)]), table, cu0).float()
    ends = [0, lens[0] + extra]
    for i, n in enumerate(lens):
        a = first[int(cu0[i]):int(cu0[i]) + n]
        assert torch.equal(a, want[ends[i]:ends[i] + n])
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    each = torch.arange(3, dtype=torch.int32, device="cuda")
    for s in range(extra):
        y = steps.decode(torch.stack([r[n + s] for r, n in zip(rows, lens)]), table, ctx, each).float()
        ctx += 1
        for i, n in enumerate(lens):
            w = want[ends[i] + n + s]
            assert float((y[i] - w).norm() / w.norm()) < 2.0 ** -3, (s, i)


def test_command(example, capsys):
    example.main(["--hidden", "512", "--heads", "8", "2", "--dim", "64", "--prompts", "130", "7", "--steps", "4"])
    assert "decode: 4 steps of 2 sequences" in capsys.readouterr().out
