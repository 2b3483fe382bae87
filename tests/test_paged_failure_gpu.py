"""Failure detection of the cache operators on the GPU, made without faulting the GPU: a bounded
wait of the kernel for many rows runs out (GDN_FAULT=stall_attention: its look-up warp publishes
nothing, for which the others wait 2 s).  Every role gives up without using what did not come, the
kernel ends, gdn_sync_status reports GDN_ERR_TIMEOUT, and the next call computes correct results.
"""
import os
import subprocess
import sys

import pytest
import torch

import gated_deltanet_linear_mixer_gb300 as gdn
from conftest import ROOT
from paged_cases import attention_excess, attention_ref, cu_of, gen, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_linear_mixer_gb300 import _build
    _build.build()
    gdn.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gdn.device_error(reset=True)
    yield
    gdn.device_error(reset=True)


def _inputs(dim, seed):
    """Few enough row tiles (32 of 128 rows) to run all at once; rows past the end hold no numbers."""
    d = gdn.KVDims(16, 4, dim, page_size=64)
    counts, kv = [256], [700]
    cache, table = make_cache(d, kv, seed)
    q = torch.randn(256, 16, dim, generator=gen(seed + 1), device="cuda").bfloat16()
    return d, cache, table, counts, kv, q


def _call(d, cache, table, counts, kv, q):
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    gdn.timing_enable(True)
    out = gdn.kv_attention(d, cache, cu_of(counts), lens, table, q, max_kv_len=kv[0])
    report = gdn.timing_report()
    gdn.timing_enable(False)
    assert "kv_prompt" in report, report
    return out


@pytest.mark.parametrize("dim", [128, 256])
def test_a_wait_that_runs_out_is_reported(monkeypatch, dim):
    d, cache, table, counts, kv, q = _inputs(dim, 5)
    monkeypatch.setenv("GDN_FAULT", "stall_attention")
    _call(d, cache, table, counts, kv, q)
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == gdn.GDN_ERR_TIMEOUT
    gdn.sync_status()  # the word was cleared by the report
    monkeypatch.delenv("GDN_FAULT")
    out = _call(d, cache, table, counts, kv, q)
    gdn.sync_status()
    assert attention_excess(d, out, *attention_ref(d, cache, table, counts, kv, q)) <= 1.0


def test_the_hook_does_not_touch_the_kernel_for_few_rows(monkeypatch):
    d, cache, table, _, kv, q = _inputs(128, 7)
    monkeypatch.setenv("GDN_FAULT", "stall_attention")
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    out = gdn.kv_attention(d, cache, cu_of([1]), lens, table, q[:1])
    gdn.sync_status()
    assert attention_excess(d, out, *attention_ref(d, cache, table, [1], kv, q[:1])) <= 1.0


@pytest.mark.parametrize("same_call", [True, False])
def test_a_wait_that_runs_out_outranks_data_out_of_range(monkeypatch, same_call):
    """An unmapped page, met first in the same call or in the one before, does not hide the timeout."""
    d, cache, table, counts, kv, q = _inputs(128, 9)
    holed = table.clone()
    holed[0, 3] = -1
    if not same_call:
        _call(d, cache, holed, counts, kv, q)
    monkeypatch.setenv("GDN_FAULT", "stall_attention")
    _call(d, cache, holed if same_call else table, counts, kv, q)
    with pytest.raises(gdn.GDNError) as e:
        gdn.sync_status()
    assert e.value.status == gdn.GDN_ERR_TIMEOUT
    monkeypatch.delenv("GDN_FAULT")
    _call(d, cache, holed, counts, kv, q)
    with pytest.raises(gdn.GDNError, match="code 40"):
        gdn.sync_status()
    gdn.sync_status()


def test_first_calls_of_a_process_may_be_captured():
    """What a process's first calls look up on the device does not get in a capture's way, and a
    replay's codes are reported."""
    code = """
import torch, gated_deltanet_linear_mixer_gb300 as gdn
from paged_cases import cu_of
d = gdn.KVDims(16, 4, 128, page_size=64, rope_dim=64)
cache = gdn.KVCache(d, *(torch.zeros(20, 4, 64, 128, dtype=torch.int8, device="cuda") for _ in "kv"),
                    *(torch.ones(20, 4, device="cuda") for _ in "kv"))
table = torch.arange(20, dtype=torch.int32, device="cuda").view(1, 20)
lens = torch.tensor([700], dtype=torch.int32, device="cuda")
new = torch.randn(300, 24, 128, device="cuda").bfloat16()
rope, cu, one = torch.ones(1280, 64, device="cuda"), cu_of([300]), cu_of([1])
ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q = gdn.kv_append(d, cache, cu, lens, table, new[:, 16:20], new[:, 20:], q=new[:, :16], rope=rope)
    a = gdn.kv_attention(d, cache, cu, lens, table, q, workspace=ws)
    b = gdn.kv_attention(d, cache, one, lens, table, q[299:], workspace=ws)
    k, v = gdn.kv_read(d, cache, one, lens - 1, table)
graph.replay()
gdn.sync_status()
assert torch.isfinite(a).all() and (a[299:].float() - b.float()).abs().max() < 0.02, (a[299:] - b).abs().max()
table.fill_(-1)
graph.replay()
try:
    gdn.sync_status()
except gdn.GDNError as e:
    assert "code 40" in str(e)
    print("reported")
"""
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, cwd=ROOT)
    assert run.returncode == 0 and run.stdout.strip() == "reported", run.stdout + run.stderr
