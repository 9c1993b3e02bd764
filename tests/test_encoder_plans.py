"""Launch plans of the encoder operators, compiled as host code."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_range_similarity_amd", "csrc")

FEW = r"""
#include <cstdio>
#include <cstdlib>
#include "embed_few_plan.h"
int main(int argc, char **argv)
{
    for (int i = 1; i < argc; ++i) {
        const long long rows = atoll(argv[i]);
        const ersj::FewPlan p = ersj::few_plan(rows);
        for (long long v = 0; v < rows; v += p.step)
            printf("%lld %lld %d %u %d %d\n", rows, v, p.own, ersj::few_groups(p, rows, v), ersj::kFewThreads,
                   ersj::kFewRows);
    }
}
"""


@pytest.fixture(scope="module")
def few_plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "few.cpp", d / "few"
    src.write_text(FEW)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def plans(rows):
        out = subprocess.run([str(exe), *map(str, rows)], check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return plans


def test_few_tokens_fit_the_largest_launch(few_plans):
    # a launch holds less than 2^32 work items along an axis; rows may number 2^31 - 2
    edges = [1, 7, 8, 9, 64, 1024, 8192, 8193, 65536, 65537, 2 ** 28, 2 ** 28 + 1, 2 ** 29 - 64, 2 ** 29 - 63, 2 ** 29,
             2 ** 29 + 1, 600000003, 2 ** 30, 2 ** 31 - 2]
    end = {}
    for rows, v, own, groups, threads, most in few_plans(edges):
        assert 1 <= own <= most
        assert 1 <= groups and groups * threads < 2 ** 32, rows
        # the launches follow each other and no workgroup is without rows
        assert v == end.get(rows, 0) and v + (groups - 1) * own < rows
        end[rows] = v + groups * own
        assert end[rows] >= rows or groups * threads == 2 ** 31
    assert sorted(end) == sorted(edges)
    assert all(e >= rows for rows, e in end.items())
