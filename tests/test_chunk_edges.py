"""The chunk operators' host side at its edges, without a device."""
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_plan_that_the_host_has_no_memory_for_is_refused():
    """Millions of pieces under a limit on the process's memory: a status, no exception through the C ABI."""
    code = """
        import ctypes, resource
        from bit_kv_cache_22_b200 import kvq
        lib = kvq.load()
        out = kvq.Chunk()
        n = (1 << 24) - 1
        counts = (ctypes.c_int32 * 1)(n)

        def plan():
            return lib.kvq_plan_prompt(1, 128, 1, 64, counts, ctypes.byref(out), None, 0)

        size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
        resource.setrlimit(resource.RLIMIT_AS, (size + (64 << 20), resource.RLIM_INFINITY))
        assert plan() == kvq.KVQ_ERR_INVALID_ARG
        assert b"memory" in lib.kvq_last_error()
        resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
        assert plan() == kvq.KVQ_OK and out.tokens == n and out.items == 1 << 23
        print("ok")
    """
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], capture_output=True, text=True, cwd=ROOT,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.returncode, r.stderr[-2000:])
