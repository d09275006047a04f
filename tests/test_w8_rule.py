"""Which kernel an int8 product takes: the rule of csrc/linear_w8.hip, line by
line, and that the GPU tests have a shape for each of its kernels, with rows of
whole 16 bytes and of odd length, plain and gated."""
import os
import re

import pytest

import test_gpu_w8
from moe_expert_ffn_route_amd import build


def up(n, d):
    return -(-n // d)


# (the line of the rule, what it means); `b(tokens, tiles)` is the line's `blocks`
RULE = [
    ("if (a.T <= 8) return launch_few<8, 1>(a, s);",
     lambda T, n, k, b: T <= 8 and "few<8, 1>"),
    ("if (a.T <= 16) return a.n_tiles < 512 ? launch_few<16, 1>(a, s) : launch_few<16, 2>(a, s);",
     lambda T, n, k, b: T <= 16 and ("few<16, 1>" if n < 512 else "few<16, 2>")),
    ("if (blocks(64, 4) <= 256 && (a.T <= 64 || a.k_tiles >= 16)) {", None),
    ("if (blocks(16, 1) <= 256) return launch_few<16, 1>(a, s);",
     lambda T, n, k, b: few(T, k, b) and b(16, 1) <= 256 and "few<16, 1>"),
    ("if (blocks(16, 2) <= 256) return launch_few<16, 2>(a, s);",
     lambda T, n, k, b: few(T, k, b) and b(16, 2) <= 256 and "few<16, 2>"),
    ("if (blocks(32, 2) <= 256) return launch_few<32, 2>(a, s);",
     lambda T, n, k, b: few(T, k, b) and b(32, 2) <= 256 and "few<32, 2>"),
    ("if (blocks(16, 4) <= 256) return launch_few<16, 4>(a, s);",
     lambda T, n, k, b: few(T, k, b) and b(16, 4) <= 256 and "few<16, 4>"),
    ("if (blocks(32, 4) <= 256) return launch_few<32, 4>(a, s);",
     lambda T, n, k, b: few(T, k, b) and b(32, 4) <= 256 and "few<32, 4>"),
    ("return launch_few<64, 4>(a, s); }",
     lambda T, n, k, b: few(T, k, b) and "few<64, 4>"),
    ("if (a.k_tiles >= 16 && blocks(128, 16) >= 512) return launch_many<8, 4>(a, s);",
     lambda T, n, k, b: k >= 16 and b(128, 16) >= 512 and "many<8, 4>"),
    ("if (a.k_tiles >= 16 && blocks(128, 8) >= 400) return launch_many<8, 2>(a, s);",
     lambda T, n, k, b: k >= 16 and b(128, 8) >= 400 and "many<8, 2>"),
    ("if (blocks(64, 8) >= 384) return launch_many<4, 2>(a, s);",
     lambda T, n, k, b: b(64, 8) >= 384 and "many<4, 2>"),
    ("if (a.k_tiles >= 16) return blocks(64, 8) >= 160 ? launch_many<4, 2, 8, 4>(a, s) : launch_many<2, 1, 8, 4>(a, s);",
     lambda T, n, k, b: k >= 16 and ("many<4, 2, 8, 4>" if b(64, 8) >= 160 else "many<2, 1, 8, 4>")),
    ("return blocks(64, 4) >= 384 ? launch_many<4, 1>(a, s) : launch_many<2, 1>(a, s);",
     lambda T, n, k, b: "many<4, 1>" if b(64, 4) >= 384 else "many<2, 1>"),
]


def few(T, k, b):
    return b(64, 4) <= 256 and (T <= 64 or k >= 16)


def kernel(T, N, K, gated):
    n, k = up(N // 2, 8) if gated else up(N, 16), up(K, 128)
    for _, rule in RULE:
        name = rule and rule(T, n, k, lambda tokens, tiles: up(T, tokens) * up(n, tiles))
        if name:
            return name, K % 16 != 0


def body():
    with open(os.path.join(build.CSRC, "linear_w8.hip")) as f:
        text = f.read()
    text = text[text.index("hipError_t launch_linear_w8("):]
    text = re.sub(r"//[^\n]*", "", text[text.index("};") + 2:text.index("}  // namespace moe")])
    return " ".join(text.split())


def test_the_rule_is_the_source_s():
    """A threshold that changes there has to change here, and then the shapes."""
    assert body() == " ".join(line for line, _ in RULE) + " }"


@pytest.mark.parametrize("gated", [False, True])
def test_every_kernel_is_tested(gated):
    names = set(re.findall(r"(?:few|many)<[0-9, ]+>", " ".join(line for line, _ in RULE)))
    assert len(names) == 14
    reached = {kernel(T, N, K, gated) for T, N, K in test_gpu_w8.EVERY}
    assert reached == {(name, odd) for name in names for odd in (False, True)}
