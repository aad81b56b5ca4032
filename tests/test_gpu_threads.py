"""Calls from several host threads at once: the header states that every function is thread-safe."""
import threading

import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import workloads as W

pytestmark = pytest.mark.gpu


def _together(jobs):
    """Runs the jobs in a thread each, from a common start; raises what the first failing one raised."""
    failed, start = [], threading.Barrier(len(jobs))

    def run(job):
        try:
            start.wait()
            job()
        except Exception as e:  # noqa: BLE001 - handed to the test
            failed.append(e)

    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert sdpa.attn_get_last_error() == 0
    if failed:
        raise failed[0]


def test_float32_forwards_of_several_head_sizes():
    """One kernel serves a range of head sizes (97 .. 128, 65 .. 96), whose blocks need different amounts of shared
    memory: a call with little must not take it from another thread's. The C calls themselves, one after the other,
    since the threads meet inside them (ctypes lets go of the interpreter's lock there)."""
    lib = sdpa.load_library()
    jobs, checks = [], []
    for D in (128, 100, 128, 100, 96, 68, 96, 68):
        inp = W.dense_bhsd(1, 1, 1, D, causal=False, dtype=torch.float32, seed=D, cfg=91)
        q, k, v = (t.cuda() for t in (inp.q, inp.k, inp.v))
        stream, out = torch.cuda.Stream(), torch.empty_like(q)
        args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, 1, 1, 1, 1, 1, D, D ** -0.5, 0, W.F32, W.BHSD,
                out.data_ptr(), None, None, stream.cuda_stream)
        torch.cuda.synchronize()

        def job(args=args, f=lib.attn_fwd):
            for _ in range(20000):
                rc = f(*args)
                if rc:
                    raise sdpa.AttnError(rc, f"attn_fwd at head size {args[10]}")

        jobs.append(job)
        checks.append((out, v, (q, k)))
    _together(jobs)
    for out, v, _ in checks:
        assert torch.equal(out, v)  # one key: its value


def test_forks_of_tables_of_many_rows():
    """Tables of more than 6,144 rows need more shared memory than a kernel has by default, each its own amount."""
    lib = sdpa.load_library()
    jobs, checks = [], []
    for rows in (8192, 6200, 8192, 6200, 7000, 6150):
        table = torch.arange(rows, dtype=torch.int32, device="cuda")
        src, ref = table.flip(0).contiguous(), torch.ones(rows, dtype=torch.int32, device="cuda")
        out, refs = torch.empty_like(table), torch.empty_like(ref)
        stream = torch.cuda.Stream()
        args = (table.data_ptr(), src.data_ptr(), ref.data_ptr(), None, rows, rows, 1, rows, out.data_ptr(),
                refs.data_ptr(), None, stream.cuda_stream)
        torch.cuda.synchronize()

        def job(args=args, f=lib.attn_cache_fork):
            for _ in range(10000):
                rc = f(*args)
                if rc:
                    raise sdpa.AttnError(rc, f"attn_cache_fork of {args[4]} rows")

        jobs.append(job)
        checks.append((out, src, refs, ref, table))
    _together(jobs)
    for out, src, refs, ref, _ in checks:
        assert torch.equal(out, src) and torch.equal(refs, ref)
