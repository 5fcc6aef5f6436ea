"""CPU checks of how bakron_matvec4 cuts a call: every call that the header allows gets a launch that
the hardware takes, on a GPU of 148 SMs (the plan is made on the host)."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from two_sided_adaptive_bakron_b200 import build as B

LIMIT = 227 * 1024            # shared memory of a block, static and dynamic together
TYPES = [torch.float32, torch.float16, torch.bfloat16, torch.int8]


@pytest.fixture(scope="module")
def bk():
    B.build()
    from two_sided_adaptive_bakron_b200 import bakron
    return bakron


def _static_bytes():
    """An upper bound of the product kernel's static shared memory: 128 bytes an array."""
    text = re.sub(r"//.*", "", open(os.path.join(B.CSRC, "matvec4.cu")).read())
    return 128 * len(re.findall(r"^(?!.*\bextern\b).*__shared__", text, flags=re.M))


def _check(bk, m, n, **kw):
    p = bk.internal_matvec4_plan(m, n, **kw)
    assert p is not None, ("refused", m, n, kw)
    assert p["smem"] + _static_bytes() <= LIMIT, (m, n, kw, p)
    rows = -(-m // 16)
    assert -(-rows // p["clusters"]) <= p["max_tiles"], (p, m)
    assert p["cluster"] * p["slice"] >= -(-n // 64) and 1 <= p["chunk"] <= kw["tokens"]
    assert p["chunk"] <= p["product_tiles"] * (2 if kw["x_dtype"] == torch.float32 else 8)
    return p


# layers, steps, codebooks and tokens whose plans fill shared memory to the last byte
@pytest.mark.parametrize("m,n,group,book,tokens,x", [
    (28672, 8192, None, False, 16, torch.bfloat16), (28672, 8192, None, False, 16, torch.float16),
    (28672, 8192, None, True, 9, torch.bfloat16), (28672, 8192, None, True, 16, torch.float16),
    (14336, 4096, None, True, 17, torch.bfloat16), (12288, 4096, None, True, 17, torch.float16),
    (28672, 4096, None, True, 16, torch.bfloat16), (32000, 4096, None, True, 16, torch.float16),
    (5120, 13824, 128, True, 16, torch.bfloat16), (3584, 18944, 128, True, 20, torch.float16),
    (8192, 8192, 128, False, 33, torch.bfloat16), (28672, 4096, None, True, 8, torch.float32),
    (4096, 11008, 128, True, 5, torch.float32), (512, 18432, 64, False, 32, torch.bfloat16),
    (4096, 5184, 64, False, 20, torch.float32), (512, 8960, 64, True, 32, torch.bfloat16)])
def test_full_plans_launch(bk, m, n, group, book, tokens, x):
    _check(bk, m, n, x_dtype=x, group_size=group, book=book, tokens=tokens)


@pytest.mark.parametrize("book", [False, True])
@pytest.mark.parametrize("x", TYPES)
def test_every_plan_launches(bk, x, book):
    for m in (1, 130, 512, 1003, 4096, 11008, 28672, 70000):
        for n in (1, 520, 4096, 5184, 8192, 8960, 14336, 18432, 28672, 49152):
            for group in (None, 32, 64, 96):
                for tokens in (1, 2, 5, 8, 9, 16, 17, 20, 32, 33, 65535):
                    if m * n >= 2 ** 31:
                        continue
                    _check(bk, m, n, x_dtype=x, group_size=group, book=book, tokens=tokens,
                           x_group_size=32 if x == torch.int8 and tokens % 2 else None)


# the longest rows, whose activations leave room for the sums of few row tiles
@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("book", [False, True])
def test_the_longest_rows_are_not_refused(bk, x, book):
    for m in (1, 20, 128, 880, 1456, 2000, 4096, 32000):
        for n in (55360, 60000, 65535, 65536):
            for group in (None, 32, 64):
                for tokens in (1, 2, 8, 16, 33, 40):
                    if m * n < 2 ** 31:
                        _check(bk, m, n, x_dtype=x, group_size=group, book=book, tokens=tokens,
                               x_group_size=32)


def test_the_limit_of_a_kernel_is_a_constant():
    """A kernel's limit on dynamic shared memory is set in one place only, to a constant: a call that
    set it to its own size could lower it between another thread's call and its launch."""
    uses = {}
    for f in sorted(os.listdir(B.CSRC)):
        text = re.sub(r"//.*", "", open(os.path.join(B.CSRC, f)).read())
        uses[f] = text.count("cudaFuncAttributeMaxDynamicSharedMemorySize")
    assert {f: k for f, k in uses.items() if k} == {"common.cuh": 1}


def test_plans_of_fp32_results_of_bf16_activations(bk):
    """With a codebook they take a table of three parts."""
    for m, n, group, tokens in [(28672, 8192, None, 16), (14336, 4096, None, 17), (5120, 13824, 128, 32),
                                (4096, 65536, 32, 40), (20, 65536, 32, 9), (1, 1, None, 1),
                                (70000, 8960, 64, 33)]:
        p = _check(bk, m, n, x_dtype=torch.bfloat16, group_size=group, book=True, tokens=tokens,
                   out_dtype=torch.float32)
        assert p["smem"] > 3 * 32768


def test_the_number_of_sms_is_asked():
    for f in sorted(os.listdir(B.CSRC)):
        text = re.sub(r"//.*", "", open(os.path.join(B.CSRC, f)).read())
        assert not re.search(r"\b148\b", text), f
