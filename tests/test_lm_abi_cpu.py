"""What the entry points of the operators around the FFN refuse: every
host-detectable error returns its code before a pointer is read or a launch
made (so these run without a GPU), and the Python binding's tensor checks."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from activation_sparse_transformer_gate_gb300 import _build

ARG, ALIGN, DTYPE, WS = -1, -2, -3, -8
A = 1 << 40          # fake, aligned "device" addresses
OFF = A + 8          # aligned to 8, not to 16
ODD = A + 2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tw.load()


def refused(fn, good, changes):
    for pos, value, code in changes:
        args = list(good)
        args[pos] = value
        assert fn(*args) == code, (fn.__name__, pos, value)


def test_embed(lib):
    ws = tw.twell_embed_workspace_size(64, 500, 128)
    assert ws >= 64 * 16
    good = [A, 8, A, 64, 500, 128, 0, 1.0, -1, A, A, None]
    common = [(0, None, ARG), (0, ODD, ALIGN), (1, 2, DTYPE), (2, None, ARG), (2, OFF, ALIGN),
              (3, 0, ARG), (3, -5, ARG), (3, (1 << 30) + 1, ARG), (4, 0, ARG),
              (4, 0x7FFFFFFF, ARG), (5, 0, ARG),
              (5, 126, ALIGN), (5, 1 << 20, ARG), (6, 5, DTYPE), (9, None, ARG), (9, OFF, ALIGN),
              (10, None, ARG), (10, ODD, ALIGN)]
    refused(lib.twell_embed_forward, good, common)
    back = good[:-1] + [A, ws, None]
    refused(lib.twell_embed_backward, back, common + [
        (11, None, WS), (11, A + 128, WS), (12, ws - 1, WS), (12, 0, WS)])
    for bad in ((0, 5, 8), (5, 0, 8), (5, 5, 0), (5, 5, 3), (5, 5, 1 << 20)):
        assert tw.twell_embed_workspace_size(*bad) == 0


def test_rmsnorm(lib):
    good = [A, A, A, 64, 128, 0, 1e-6, A, A, A, A, A, None]
    f = lib.twell_add_rmsnorm_forward
    refused(f, good, [
        (0, None, ARG), (0, OFF, ALIGN), (1, OFF, ALIGN), (2, None, ARG), (2, OFF, ALIGN),
        (3, 0, ARG), (3, (1 << 30) + 1, ARG), (4, 0, ARG), (4, 130, ALIGN), (4, 8192, ARG),
        (5, 2, DTYPE), (6, -1.0, ARG),
        (6, float("nan"), ARG), (7, None, ARG), (7, OFF, ALIGN), (8, OFF, ALIGN), (9, OFF, ALIGN),
        (10, None, ARG), (10, ODD, ALIGN), (11, ODD, ALIGN)])
    assert f(A, A, A, 64, 128, 0, 1e-6, A, None, None, A, A, None) == ARG   # no output
    assert f(A, None, A, 64, 136, 1, 1e-6, A, None, A, A, A, None) == ALIGN  # 8-bit rows of 136
    ws = tw.twell_add_rmsnorm_workspace_size(64, 128)
    assert ws > 0
    good = [A, A, A, A, A, 64, 128, 1, A, A, A, ws, None]
    refused(lib.twell_add_rmsnorm_backward, good, [
        (0, None, ARG), (0, OFF, ALIGN), (1, None, ARG), (2, None, ARG), (3, None, ARG),
        (3, OFF, ALIGN), (4, OFF, ALIGN), (5, 0, ARG), (6, 100, ALIGN), (6, 8200, ARG), (7, 9, DTYPE),
        (8, None, ARG), (8, OFF, ALIGN), (9, None, ARG), (9, ODD, ALIGN), (10, None, WS),
        (10, A + 16, WS), (11, ws - 1, WS)])
    for bad in ((0, 128), (4, 0), (4, 10), (4, 16384)):
        assert tw.twell_add_rmsnorm_workspace_size(*bad) == 0


def test_q8(lib):
    refused(lib.twell_q8_quantize, [A, 4, 64, 0, A, A, None], [
        (0, None, ARG), (0, OFF, ALIGN), (1, 0, ARG), (2, 0, ARG), (2, 40, ALIGN), (3, 3, DTYPE),
        (4, None, ARG), (4, OFF, ALIGN), (5, None, ARG), (5, ODD, ALIGN)])
    ws = tw.twell_q8_workspace_size(10, 20, 64)
    good = [A, A, A, A, A, 10, 20, 64, 1, A, A, A, max(ws, 1), None]
    refused(lib.twell_q8_matmul, good, [
        (0, None, ARG), (0, OFF, ALIGN), (1, None, ARG), (1, ODD, ALIGN), (2, None, ARG),
        (2, OFF, ALIGN), (3, None, ARG), (3, ODD, ALIGN), (4, ODD, ALIGN), (5, 0, ARG), (6, 0, ARG),
        (5, (1 << 30) + 1, ARG), (6, (1 << 30) + 1, ARG), (7, 0, ARG), (7, 24, ALIGN),
        (7, 65552, ARG), (8, 4, DTYPE), (9, None, ARG), (9, OFF, ALIGN),
        (10, None, ARG), (10, ODD, ALIGN)])
    ws = tw.twell_q8_workspace_size(300, 20, 64)      # many rows: scratch for the widened rows
    assert ws >= 300 * 64 * 2
    good = [A, A, A, A, A, 300, 20, 64, 1, A, A, A, ws, None]
    refused(lib.twell_q8_matmul, good, [(11, None, WS), (11, A + 64, WS), (12, ws - 1, WS)])
    for bad in ((0, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 20), (1, 1, 65552)):
        assert tw.twell_q8_workspace_size(*bad) == 0


def test_distill(lib):
    good = [A, 512, A, A, A, 4, 500, 8, 0, 1.0, A, A, A, A, None]
    refused(lib.twell_distill_forward, good, [
        (0, None, ARG), (0, OFF, ALIGN), (1, 499, ARG), (2, None, ARG), (2, ODD, ALIGN),
        (3, None, ARG), (4, ODD, ALIGN), (5, 0, ARG), (5, (1 << 30) + 1, ARG), (6, 0, ARG),
        (7, 0, ARG), (7, 257, ARG),
        (8, 7, DTYPE), (9, 0.0, ARG), (9, -1.0, ARG), (9, float("nan"), ARG), (9, float("inf"), ARG),
        (10, None, ARG), (11, None, ARG), (11, A + 4, ALIGN), (12, OFF, ALIGN), (13, None, ARG)])
    back = [A, 512, A, A, A, A, 4, 500, 8, 0, 1.0, A, A, None]
    refused(lib.twell_distill_backward, back, [
        (0, None, ARG), (4, None, ARG), (5, None, ARG), (10, 1e-5, ARG), (11, None, ARG),
        (11, OFF, ALIGN), (12, None, ARG)])


def test_read_status(lib):
    assert lib.twell_read_status(None, None) == ARG


def test_binding_checks_tensors(lib):
    """Type, size and place of a tensor are checked before the call."""
    cpu = torch.zeros(64, 128)

    def code(*args, fn=tw.twell_add_rmsnorm_forward):
        with pytest.raises(tw.TwellError) as e:
            fn(*args, stream=0)
        return e.value.code

    rest = (A, 64, 128, tw.TWELL_F32, 1e-6, A, A, A, A, A)
    assert code(cpu, A, *rest) == ARG                       # not on the GPU
    assert code(cpu.bfloat16(), A, *rest) == DTYPE
    assert code(A, A, A, 64, 128, 9, 1e-6, A, A, A, A, A) == DTYPE
    assert code(torch.zeros(63, 128), A, *rest) == ARG
    z = torch.zeros(4, 512)
    assert code(z[:, :500], 512, A, A, A, 4, 500, 8, tw.TWELL_F32, 1.0, A, A, A, A,
                fn=tw.twell_distill_forward) == ARG          # not on the GPU
    assert code(torch.zeros(64, dtype=torch.int16), A, 64, 500, 128, 0, 1.0, -1, A, A,
                fn=tw.twell_embed_forward) == DTYPE
    with pytest.raises(AttributeError):
        tw.no_such_operator
    # what is neither a tensor, nor a pointer, nor a number raises as such
    with pytest.raises(TypeError):
        tw.twell_add_rmsnorm_forward("x", A, *rest, stream=0)
    with pytest.raises(TypeError):
        tw.twell_add_rmsnorm_forward(A, A, A, 64, 128, tw.TWELL_F32, "eps", A, A, A, A, A, stream=0)
    assert code(A, A, A, 1 << 40, 128, tw.TWELL_F32, 1e-6, A, A, A, A, A) == ARG
    assert code(A, A, A, A, A, 64, 128, tw.TWELL_F32, A, A, torch.zeros(10), 1 << 20,
                fn=tw.twell_add_rmsnorm_backward) == WS


@pytest.mark.parametrize("M,N,K", [(5, 1000, 16384), (8, 128, 65536), (16, 512, 16384),
                                   (32, 1000, 8192), (48, 1024, 8192), (64, 1024, 8192),
                                   (64, 2048, 4096), (64, 128, 65536)])
def test_long_sums_of_few_columns_leave_the_fragments(lib, M, N, K):
    """Few columns with a long k are multiplied where clusters share k, which needs the widened rows
    of a as scratch."""
    assert tw.twell_q8_workspace_size(M, N, K) >= M * K * 2
    assert tw.twell_q8_workspace_size(M, N, 1024) == 0


def test_pair_counts_are_in_the_test_variants_only(lib):
    assert not hasattr(lib, "twell_test_q8_pairs")
    _build.build(variants=("hooks", "timeout"))
    for variant in ("hooks", "timeout"):
        assert hasattr(tw.load(_build.lib_path(variant)), "twell_test_q8_pairs")
