"""The last CTA of a split request copies partial results that other CTAs stored: what orders their plain stores before its bulk
copies, and merges over and over with other partials in the same memory."""
import os
import re

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4, KVCache, build


def test_partials_are_ordered_before_the_copies():
    """After the acquire and before the copy, the copying thread orders global memory between the proxies."""
    text = open(os.path.join(build.CSRC, "common.cuh")).read()
    body = text[text.index("__device__ bool merge_partial("):]
    body = re.sub(r"//[^\n]*", "", body[:body.index("\n}\n")])
    acquire, copy = body.index("atomic_add_acq_rel("), body.index("bulk_g2s(")
    assert acquire < body.index("fence_proxy_async_global();") < copy
    assert 'fence.proxy.async.global;' in text[text.index("void fence_proxy_async_global()"):][:120]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["int4", "bf16", "window"])
def test_merges_one_after_the_other(kind):
    """Queries in turn: a partial of the call before would show."""
    lengths, hkv, gqa = [9000, 20000, 700, 33, 12345], 4, 8
    pages = sum(-(-n // 64) for n in lengths)
    c = KVCache(fmt=OSCAR_FORMAT_INT4 if kind == "int4" else OSCAR_FORMAT_BF16, n_q_heads=hkv * gqa, n_kv_heads=hkv, group=32,
                max_requests=len(lengths), max_pages=pages, max_pages_per_request=pages)
    slots = [c.alloc() for _ in lengths]
    c.reserve(slots, lengths)
    g = torch.Generator(device="cuda").manual_seed(1)
    c.append(0, *(torch.randn(sum(lengths), hkv, 128, generator=g, device="cuda").bfloat16() for _ in range(2)))
    c.commit()
    qs = [torch.randn(len(lengths), hkv * gqa, 128, generator=g, device="cuda").bfloat16() for _ in range(4)]
    if kind == "window":
        c.plan_window(slots)
        run = c.attend_window
    else:
        c.plan(slots, max_split_pages=7)
        run = c.decode
    want = []
    for q in qs:
        want.append(run(0, q))
        torch.cuda.synchronize()
    wrong = torch.zeros((), dtype=torch.long, device="cuda")
    for i in range(400):
        out = run(0, qs[i % 4])
        wrong += (out != want[i % 4]).sum()
    assert int(wrong) == 0 and c.status() == (0, 0)
