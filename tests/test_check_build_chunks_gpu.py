"""The chunk operators under the bounds-check build (libkvq_check.so, KVQ_LIBRARY=check) on a GPU, in child
processes: their suites pass, and bounded waits of the attention kernels that run out are reported, leave
the other CTAs' outputs alone and the context, the tensor memory with it, usable."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_chunk_suites_under_the_bounds_check_build():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_chunk_gpu.py", "tests/test_chunk_edges_gpu.py",
                        "-k", "not prompt_attention and not hardly_weigh and not hundred"],
                       capture_output=True, text=True, env=dict(os.environ, KVQ_LIBRARY="check"), cwd=ROOT, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:]
    assert " passed" in r.stdout


COMMON = """
    import torch
    from bit_kv_cache_22_b200 import kvq
    import chunk_testlib as ct
    assert kvq.check_build() and kvq.library_path().endswith("libkvq_check.so")
    lib = kvq.load()

    def stalls(call, check):
        for tile in (1, 2, 4):
            assert lib.kvq_debug_set_attention_stall(tile) == kvq.KVQ_OK
            call()
            try:
                check()
                raise SystemExit(f"no wait gave up at tile {tile}")
            except kvq.KVQError as e:
                assert e.status == kvq.KVQ_ERR_DEVICE_CHECK and "0x1" in str(e), e
            assert lib.kvq_debug_set_attention_stall(0) == kvq.KVQ_OK
            check()                                 # cleared
            yield tile
"""

PROMPT = COMMON + """
    lens, hq, hkv, d = [700, 90, 300], 8, 2, 128
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(sum(lens), h, d, generator=gen).to(torch.bfloat16) for h in (hq, hkv, hkv))
    dev = [x.cuda() for x in (q, k, v)]
    plan = kvq.plan_prompt(lens, hq, hkv, d)
    want = kvq.prompt_attention(plan, *dev)
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        ct.check_attention(want[rows], *ct.attend(ct.wide(q[rows]), ct.wide(k[rows]).transpose(1, 0, 2),
                                                  ct.wide(v[rows]).transpose(1, 0, 2), 0), n, q.dtype, False)
        at += n
    out = torch.empty_like(want)

    def call():
        out.fill_(9.0)
        kvq.prompt_attention(plan, *dev, out=out)

    for tile in stalls(call, plan.check_device):
        lost = (out == 9.0).all(-1)                 # the first CTA's piece: 64 tokens x the first kv head's queries
        assert lost.sum() == (700 - 640) * 4 and lost[640:700, :4].all(), lost.sum()
        assert torch.equal(out[~lost], want[~lost])
        assert torch.equal(kvq.prompt_attention(plan, *dev), want)
    print("ok")
"""

CHUNK = COMMON + """
    counts = {counts}
    p = ct.Pair(4, 8, 2, 128, 32, 32, 128, 2, False, torch.bfloat16, 2048, 128)
    p.append([1500, 200, 700, 0])
    plan, _, _ = p.append(counts)
    q = p.new(plan.tokens, 8)
    dq = q.cuda()
    want = p.check_attention(plan, q)
    out = torch.empty_like(want)

    def call():
        out.fill_(9.0)
        p.cache.chunk_attention(plan, dq, out=out)

    for tile in stalls(call, p.cache.check_device):
        if plan.chunk.merges == 0:
            lost = (out == 9.0).all(-1)
            assert 0 < lost.sum() <= 64 * 4
            assert torch.equal(out[~lost], want[~lost])
        assert torch.equal(p.cache.chunk_attention(plan, dq), want)
    p.check_state()
    print("ok")
"""


@pytest.mark.parametrize("code", [PROMPT, CHUNK.replace("{counts}", "[2, 3, 0, 1]"), CHUNK.replace("{counts}", "[200, 90, 60, 0]")],
                         ids=["prompt", "narrow", "wide"])
def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable(code):
    env = dict(os.environ, KVQ_LIBRARY="check", PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], capture_output=True, text=True, env=env, cwd=ROOT,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.stdout[-2000:], r.stderr[-3000:])
