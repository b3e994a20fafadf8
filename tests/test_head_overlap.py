"""When two tensors of an attention call share an element: the host's rule (head_tensor.hpp,
built for the CPU) against the sets of their elements."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# stdin: two layouts (tokens heads head_dim token_stride head_stride) and the second's offset,
# a line each; stdout: 1 or 0 for each line
PROGRAM = r"""
#include <cstdio>
#include "head_tensor.hpp"
using namespace fp8k;
int main()
{
    auto layout = [](HeadLayout& h) {
        long long t, n, d, row, head;
        if (scanf("%lld %lld %lld %lld %lld", &t, &n, &d, &row, &head) != 5) return false;
        h.tokens = t, h.heads = n, h.d = d, h.head = n == 1 ? 0 : head, h.row = kernel_row(t, d, row);
        return true;
    };
    HeadLayout a, b;
    long long off;
    while (layout(a) && layout(b) && scanf("%lld", &off) == 1) puts(share_element(a, b, off) ? "1" : "0");
}
"""


@pytest.fixture(scope="module")
def shared(tmp_path_factory):
    where = tmp_path_factory.mktemp("head_overlap")
    src, exe = where / "share.cpp", where / "share"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "fp8_precision_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, (*a, *b, off))) for a, b, off in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(cases)
        return [o == "1" for o in out]

    return ask


def elements(layout, at):
    tokens, heads, d, row, head = layout
    i, j, k = np.arange(tokens)[:, None, None], np.arange(heads)[None, :, None], np.arange(d)[None, None, :]
    return set((at + i * row + j * head + k).reshape(-1).tolist())


def truth(a, b, off):
    return bool(elements(a, 0) & elements(b, off))


def test_slices_of_one_tensor_interleave(shared):
    """[tokens, heads, 3, d], [tokens, 3, heads, d], [heads, 3, tokens, d] and a projection with
    fewer key heads: the three slices are apart, in any order."""
    t, h, d = 7, 4, 16
    by_layout = {"head, 3, d": ((t, h, d, 3 * h * d, 3 * d), d), "3, head, d": ((t, h, d, 3 * h * d, d), h * d),
                 "head major": ((t, h, d, d, 3 * t * d), t * d), "one token": ((1, h, d, d, 3 * d), d),
                 "one head": ((t, 1, d, 3 * d, 5), d), "more heads than a row holds": ((t, 3, d, 2 * d, 2 * t * d), d)}
    for name, (layout, step) in by_layout.items():
        n = 2 if name.startswith("more") else 3
        cases = [(layout, layout, step * (j - i)) for i in range(n) for j in range(n) if i != j]
        assert not any(truth(*c) for c in cases), name
        assert not any(shared(cases)), name
    q, k = (t, 4, d, 8 * d, d), (t, 2, d, 8 * d, d)
    assert shared([(q, k, 4 * d), (q, k, 6 * d), (k, k, 2 * d), (k, q, -4 * d)]) == [False] * 4


def test_sharing_is_seen(shared):
    t, h, d = 7, 4, 16
    inter = (t, h, d, 3 * h * d, 3 * d)
    cases = [(inter, inter, 0), (inter, inter, 3 * d), (inter, inter, 8), (inter, inter, d - 8), (inter, inter, 2 * d + 8),
             (inter, inter, 3 * h * d), (inter, (t, h, d, 3 * h * d, d), 0), ((1, h, d, d, 3 * d), (1, h, d, d, 3 * d), 6 * d),
             ((t, h, d, d, 3 * t * d), (t, h, d, d, 3 * t * d), t * d - 8)]
    assert all(truth(*c) for c in cases)
    assert all(shared(cases))


def test_against_the_sets_of_elements(shared):
    """Never "apart" where an element is shared; with equal strides the rule is exact."""
    rng = np.random.default_rng(1)
    cases = []
    for _ in range(4000):
        d = 8 * int(rng.integers(1, 3))
        row, head = (d + 8 * int(rng.integers(0, 14)) for _ in range(2))
        other = rng.random() < 0.3
        one = lambda r, c: (int(rng.integers(1, 6)), int(rng.integers(1, 6)), d, r, c)
        a = one(row, head)
        b = one(row + 8 * int(rng.integers(0, 2)) if other else row, head + 8 * int(rng.integers(0, 2)) if other else head)
        cases.append((a, b, 8 * int(rng.integers(-60, 60))))
    said = shared(cases)
    for (a, b, off), yes in zip(cases, said):
        real = truth(a, b, off)
        assert yes or not real, (a, b, off)
        if a[3:] == b[3:]:
            assert yes == real, (a, b, off)
