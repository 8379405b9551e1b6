"""How many tokens a CTA of the store into 8-bit pages looks at, read from the source.

A CTA of 16 takes up to 16 single tokens one after another (some 40 us), so steps in
which single tokens stand beside a prompt have to get a CTA for every token; long
prompts are faster with 16."""
import re

import pytest

from test_launch_order_host import source

CTAS = 304  # resident on a GPU of 152 SMs


def single(ql):
    rule = re.search(r"const bool single = ([^;]+);", source("paged_store_e4m3.cu")).group(1)
    for a, b in (("p.m.N", str(sum(ql))), ("p.m.A", str(len(ql))), ("ctas", str(CTAS)), ("||", " or ")):
        rule = rule.replace(a, b)
    return eval(re.sub(r"(\d)ll\b", r"\1", rule))


@pytest.mark.parametrize("ql", [[1] * 32, [1] * 2048, [1] * 63 + [1100], [1] * 20 + [400], [1] * 22 + [40, 100, 200, 300, 400, 512],
                                [1] * 31 + [2048], [1] * 15 + [2048], [1] * 30 + [512] * 8, [4] * 512, [24] * 32])
def test_a_cta_for_every_token(ql):
    assert single(ql)


@pytest.mark.parametrize("ql", [[1024] * 16, [301, 700, 1237], [1024] * 16 + [1] * 16, [2048] * 4, [256] * 16])
def test_a_cta_for_sixteen_tokens(ql):
    assert not single(ql)
