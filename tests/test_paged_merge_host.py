"""The order of memory around the merge of a small call's parts, read from the
source: one lane counts the parts with an acquiring atomic, and a shuffle, which
tells the others what it found, orders nothing."""
import re

from test_launch_order_host import source


def test_the_warp_synchronises_between_the_count_and_the_merge():
    text = source("paged_attention.cu")
    at = text.index("atomic_add_acq_rel_gpu(count")
    between = text[at:text.index("merge_small<D, F16>(", at)]
    shuffle = between.index("__shfl_sync")
    assert re.search(r"__syncwarp\(\)|__threadfence\(\)", between[shuffle:]), \
        "the merging lanes read other CTAs' parts behind a shuffle alone"
