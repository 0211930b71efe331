"""Shared helpers of the tests of the operators around the FFN: inputs, call
wrappers that allocate outputs, and the half-ulp allowance of an output type."""
import torch

import activation_sparse_transformer_gate_gb300 as tw

DT = {"bf16": (torch.bfloat16, tw.TWELL_BF16), "f32": (torch.float32, tw.TWELL_F32)}
U = 2.0 ** -24  # unit roundoff of fp32


def setup():
    import pytest
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw._build.build()
    tw.load()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def scratch(n):
    """A workspace filled with NaN bit patterns: nothing may depend on what it held."""
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda"), n


def empty(*shape, dtype=torch.float32):
    """An output buffer filled with NaN (or the least int8)."""
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t.fill_(float("nan")) if dtype.is_floating_point else t.fill_(-128)


def half_ulp(ref, dtype):
    """Half a unit in the last place of the output type at |ref| (64-bit tensor)."""
    a = ref.abs()
    e = torch.floor(torch.log2(a.clamp_min(1e-37)))
    return torch.where(a > 0, torch.exp2(e - (7 if dtype == "bf16" else 23) - 1), 0.0)


def check(got, ref, bound, dtype, name):
    """|got - ref| <= bound + half an ulp of the stored type, elementwise; infinities and NaN
    where the reference has them."""
    got = got.detach().double().cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), name
    assert torch.equal(got[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)]), name
    z = torch.zeros_like(ref)
    d = torch.where(fin, (got - ref).abs(), z)
    # (a value that rounds up to the next binade has twice the ulp of ref)
    allow = torch.where(fin, bound + half_ulp(torch.where(fin, ref.abs() + bound, z), dtype), z)
    worst = (d - allow).max().item() if d.numel() else 0.0
    assert worst <= 0, f"{name}: beyond the bound by {worst:.3e}, |d| max {d.max().item():.3e}"
